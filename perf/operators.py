"""What is measured of the prompt side of the library: requests' pages and
slots laid out on the GPU (tables), new token rows written into the paged
cache by slot (append), cached latents expanded to per-head keys and values
(expand), and attention of ragged chunks of new tokens over them (prefill).

``run`` computes an operator in elementary torch operations, or, where ``own``
is true, through the library's entry points.
"""

import math
import random

import torch

own = False

PAGE = 64
ROPE_BASE = 10000.0
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of the MLA serving batch: one new token for each of 64 requests
        dict(name="tables_decode_64", op="tables", batch=64, cached_lo=4096, cached_hi=32768, new_lo=1, new_hi=1, lens=1),
        # a batch of fresh prompts (the GQA batch's lengths): pages for 150 thousand tokens
        dict(name="tables_prompts_32", op="tables", batch=32, cached_lo=0, cached_hi=0, new_lo=1024, new_hi=8192, lens=2),
        # the rows of one decode step of 64 sequences, latent cache
        dict(name="append_mla_64", op="append", kind="mla", tokens=64, lens=3),
        # the rows of a prompt step, latent cache, an odd number of tokens
        dict(name="append_mla_20011", op="append", kind="mla", tokens=20011, lens=4),
        # a prompt's keys and values quantised into the fp8 cache (8 KV heads x 128), keys turned
        dict(name="append_fp8_9001", op="append", kind="gqa_fp8", tokens=9001, lens=5),
        # ragged prompts' latents (512 wide) to 128 heads' keys and values
        dict(name="expand_mla_4x", op="expand", heads=128, groups=1, d_c=512, d_k=128, d_v=128, batch=4, lo=1024, hi=8192, lens=6),
        # one 16K prompt of GLA-2: two 256-wide latents, 64 heads each
        dict(name="expand_gla_16k", op="expand", heads=128, groups=2, d_c=256, d_k=128, d_v=128, batch=1, lo=16384, hi=16384, lens=7),
        # the smallest attention call: two 512-token prompts, 8 heads of 64 + 16
        dict(name="prefill_tiny_2x512", op="prefill", heads=8, kv_heads=8, d_nope=64, d_rope=16, d_v=64, batch=2, q_lo=512, q_hi=512,
             past_lo=0, past_hi=0, causal=True, lens=8),
        # many short ragged prompts in one step
        dict(name="prefill_short_32x", op="prefill", heads=32, kv_heads=32, d_nope=128, d_rope=64, d_v=128, batch=32, q_lo=1, q_hi=1024,
             past_lo=0, past_hi=0, causal=True, lens=9),
        # grouped heads, no rope part, keys and values token by token as projected (the GQA batch's lengths)
        dict(name="prefill_gqa_4x", op="prefill", heads=32, kv_heads=8, d_nope=128, d_rope=0, d_v=128, batch=4, q_lo=1024, q_hi=8192,
             past_lo=0, past_hi=0, causal=True, lens=10),
        # chunks of a long prompt whose first 16K tokens are cached (chunked prefill)
        dict(name="prefill_mla_chunk", op="prefill", heads=128, kv_heads=128, d_nope=128, d_rope=64, d_v=128, batch=2, q_lo=999, q_hi=1024,
             past_lo=15000, past_hi=16384, causal=True, lens=11),
        # one 8K prompt, 128 heads of 128 + 64: the largest call
        dict(name="prefill_mla_8k", op="prefill", heads=128, kv_heads=128, d_nope=128, d_rope=64, d_v=128, batch=1, q_lo=8192, q_hi=8192,
             past_lo=0, past_hi=0, causal=True, lens=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "expand", "prefill", "prefill"])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        batch = log_int(rng, 1, 512)
        hi = log_int(rng, 1, 8192 if batch <= 32 else 512)
        past = rng.choice([0, log_int(rng, 1, 32768)])
        return dict(op=op, batch=batch, cached_lo=0, cached_hi=past, new_lo=rng.choice([0, 1]), new_hi=hi, lens=lens)
    if op == "append":
        return dict(op=op, kind=rng.choice(["mla", "gla", "gqa", "gqa_fp8"]), tokens=log_int(rng, 1, 20011), lens=lens)
    if op == "expand":
        groups, d_c = rng.choice([(1, 512), (2, 256), (1, 256), (4, 128), (1, 64)])
        width = rng.choice([64, 128])
        heads = groups * rng.choice([4, 8, 16, 32])
        batch = rng.choice([1, 2, 3, 5, 8])
        return dict(op=op, heads=heads, groups=groups, d_c=d_c, d_k=width, d_v=rng.choice([width, 128]), batch=batch, lo=0,
                    hi=log_int(rng, 16, 16384 // batch), lens=lens)
    kv_heads = rng.choice([2, 4, 8, 16, 32])
    heads = kv_heads * rng.choice([1, 1, 4])
    d_nope, d_rope, d_v = rng.choice([(128, 64, 128), (128, 64, 128), (128, 0, 128), (64, 0, 64), (64, 16, 64)])
    batch = rng.choice([1, 2, 3, 7, 16])
    q_hi = log_int(rng, 1, 8192 // batch)
    past = rng.choice([0, 0, log_int(rng, 1, 16384 // batch)])
    causal = rng.random() < 0.8
    # no more pairs than the largest listed case works off
    while heads * batch * q_hi * (q_hi / 2 + past if causal else q_hi + past) > 128 * 8192 * 4096:
        q_hi //= 2
    return dict(op=op, heads=heads, kv_heads=kv_heads, d_nope=d_nope, d_rope=d_rope, d_v=d_v, batch=batch, q_lo=rng.choice([0, 1, q_hi]),
                q_hi=q_hi, past_lo=0, past_hi=past, causal=causal, lens=lens)


def lengths(case, lo, hi, salt):
    """The batch's lengths: of the case, not of the inputs' seed. The first request has something in it."""
    rng = random.Random(case["lens"] * 1009 + salt)
    got = [rng.randint(lo, hi) for _ in range(case["batch"])]
    return [max(got[0], min(hi, 1))] + got[1:]


def pages_of(n):
    return (n + PAGE - 1) // PAGE


def starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)


# ------------------------------------------------------------------- the inputs

#: kind: (variant, heads, kv heads / groups, nope or latent width, rope width)
CACHES = {"mla": ("mla", 128, 1, 512, 64), "gla": ("gla", 128, 2, 256, 64), "gqa": ("gqa", 32, 8, 128, 0), "gqa_fp8": ("gqa", 32, 8, 128, 0)}
K_SCALE, V_SCALE = 0.5, 2.0


def normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "tables":
        cached = lengths(case, case["cached_lo"], case["cached_hi"], 1)
        new = lengths(case, case["new_lo"], case["new_hi"], 2)
        held = [pages_of(c) for c in cached]
        need = [pages_of(c + n) for c, n in zip(cached, new)]
        used = sum(held)
        num_pages = sum(need) + max(1, sum(need) // 100)
        perm = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
        mpps = max(pages_of(case["cached_hi"] + case["new_hi"]), 1)
        # held pages come off the front of the permutation, the rest is the free list
        index = torch.full((case["batch"], mpps), -1, dtype=torch.int64)
        at = 0
        for b, n in enumerate(held):
            index[b, :n] = torch.arange(at, at + n)
            at += n
        index = index.to(DEV)
        st["block_table"] = torch.where(index >= 0, perm[index.clamp(min=0)], -1).to(torch.int32)
        st["free_pages"] = torch.cat([perm[used:], torch.full((used,), -1, dtype=torch.int32, device=DEV)])
        st["free_count"] = torch.tensor([num_pages - used], dtype=torch.int32, device=DEV)
        st["cached"] = torch.tensor(cached, dtype=torch.int32, device=DEV)
        st["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        # room for the step's tokens, padded as a captured step would be
        st["max_tokens"] = max(64, (sum(new) + 63) // 64 * 64)
        st["num_pages"] = num_pages
    elif case["op"] == "append":
        _, _, kv, dn, dr = CACHES[case["kind"]]
        n = case["tokens"]
        num_pages = pages_of(n) + pages_of(n) // 8 + 2
        if case["kind"] in ("mla", "gla"):
            st["new_kv"] = normal(gen, n, kv * dn + dr)
            st["cache"] = normal(gen, num_pages, PAGE, kv * dn + dr)
        else:
            st["new_kv"] = normal(gen, n, 2, kv, dn)
            st["cache"] = normal(gen, num_pages, 2, PAGE, kv, dn)
            if case["kind"] == "gqa_fp8":
                st["cache"] = st["cache"].to(torch.float8_e4m3fn)
        # runs of tokens in scattered pages, in order inside each page
        perm = torch.randperm(num_pages, generator=gen, device=DEV)[:pages_of(n)]
        st["slots"] = (perm[:, None] * PAGE + torch.arange(PAGE, device=DEV)).reshape(-1)[:n].to(torch.int32)
        first = random.Random(case["lens"]).randrange(0, 32768)
        st["pos"] = torch.arange(first, first + n, device=DEV, dtype=torch.int32)
        st["num_pages"] = num_pages
    elif case["op"] == "expand":
        lens = lengths(case, case["lo"], case["hi"], 3)
        H, G, dc = case["heads"], case["groups"], case["d_c"]
        need = [pages_of(x) for x in lens]
        num_pages = sum(need) + 2
        st["cache"] = normal(gen, num_pages, PAGE, G * dc + 64)
        perm = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
        mpps = max(need + [1])
        index = torch.zeros((case["batch"], mpps), dtype=torch.int64)
        at = 0
        for b, n in enumerate(need):
            index[b, :n] = torch.arange(at, at + n)
            at += n
        st["block_table"] = perm[index.to(DEV)].contiguous()
        st["w_uk"] = normal(gen, H, case["d_k"], dc, scale=dc ** -0.5)
        st["w_uv"] = normal(gen, H, dc, case["d_v"], scale=dc ** -0.5)
        st["kv_start"] = starts(lens).to(DEV)
        st["lens"], st["total"], st["num_pages"], st["mpps"] = lens, sum(lens), num_pages, mpps
    else:
        q = lengths(case, case["q_lo"], case["q_hi"], 4)
        k = [a + b for a, b in zip(q, lengths(case, case["past_lo"], case["past_hi"], 5))]
        H, KH = case["heads"], case["kv_heads"]
        tq, tk = max(sum(q), 1), max(sum(k), 1)
        st["q_nope"] = normal(gen, tq, H, case["d_nope"])
        st["q_rope"] = normal(gen, tq, H, case["d_rope"]) if case["d_rope"] else None
        st["k_rope"] = normal(gen, tk, case["d_rope"]) if case["d_rope"] else None
        if case["d_rope"]:      # expanded keys and values: one block a head
            st["k"] = normal(gen, KH, tk, case["d_nope"])
            st["v"] = normal(gen, KH, tk, case["d_v"])
        else:                   # projected token by token
            st["k"] = normal(gen, tk, KH, case["d_nope"]).transpose(0, 1)
            st["v"] = normal(gen, tk, KH, case["d_v"]).transpose(0, 1)
        st["q_start"], st["kv_start"] = starts(q).to(DEV), starts(k).to(DEV)
        st["q_lens"], st["k_lens"] = q, k
        st["scale"] = (case["d_nope"] + case["d_rope"]) ** -0.5
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return {"tables": own_tables, "append": own_append, "expand": own_expand, "prefill": own_prefill}[op](st)
    return {"tables": plain_tables, "append": plain_append, "expand": plain_expand, "prefill": plain_prefill}[op](st)


def own_tables(st):
    from shared_kv_caches_b200 import kvattn as K
    return K.build_tables_tensors(st["cached"], st["new"], st["free_pages"], st["free_count"], st["block_table"], st["max_tokens"])


def own_append(st):
    from shared_kv_caches_b200 import kvattn as K
    variant, heads, kv, dn, dr = CACHES[st["case"]["kind"]]
    fp8 = st["case"]["kind"] == "gqa_fp8"
    p = K.make_params(1, heads, kv, dn, dr, st["num_pages"], st["num_pages"], 0, cache_dtype=K.KVATTN_CACHE_FP8_E4M3 if fp8 else K.KVATTN_CACHE_BF16,
                      k_scale=K_SCALE, v_scale=V_SCALE)
    K.append_slots_tensor(K.VARIANTS[variant], p, st["new_kv"], st["pos"], st["slots"], st["cache"], ROPE_BASE)
    return st["cache"]


def own_expand(st):
    from shared_kv_caches_b200 import kvattn as K
    c = st["case"]
    p = K.make_params(c["batch"], c["heads"], c["groups"], c["d_c"], 64, st["mpps"], st["num_pages"], 0)
    return K.expand_kv_tensors(K.KVATTN_MLA if c["groups"] == 1 else K.KVATTN_GLA, p, st["cache"], st["block_table"], st["kv_start"], st["w_uk"],
                               st["w_uv"], st["total"])


def own_prefill(st):
    from shared_kv_caches_b200 import kvattn as K
    return K.prefill_tensors(st["q_nope"], st["q_rope"], st["k"], st["k_rope"], st["v"], st["q_start"], st["kv_start"], st["scale"],
                             causal=st["case"]["causal"])


def plain_tables(st):
    """Pages for every request's new tokens off the top of the free list, in
    request order; each new token's position and slot; the chunks' starts."""
    cached, new, table = st["cached"].long(), st["new"].long(), st["block_table"]
    total = cached + new
    held, need = (cached + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
    first = (need - held).cumsum(0) - (need - held)          # pages taken by the requests before
    cols = torch.arange(table.shape[1], device=DEV)
    fresh = (cols >= held[:, None]) & (cols < need[:, None])
    taken = st["free_count"].long() - 1 - (first[:, None] + cols - held[:, None])
    table.copy_(torch.where(fresh, st["free_pages"][taken.clamp(0, st["free_pages"].numel() - 1)], table))
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    q_start, kv_start = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, total.cumsum(0)])
    t = torch.arange(st["max_tokens"], device=DEV)
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    live = b < cached.numel()
    b = b.clamp(max=cached.numel() - 1)
    pos = torch.where(live, cached[b] + t - q_start[b], 0)
    page = table[b, (pos // PAGE).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live, page * PAGE + pos % PAGE, -1)
    left = st["free_count"].long() - (need - held).sum()
    return dict(block_table=table, seq_lens=total.int(), free_left=left.int(), q_start=q_start.int(), kv_start=kv_start.int(), pos=pos.int(), slots=slots.int())


def turn(x, pos):
    """Rotary embedding of consecutive pairs of x [..., d] at pos, in 64 bits."""
    d = x.shape[-1]
    angle = pos.double()[:, None] * ROPE_BASE ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    while angle.dim() < x.dim():
        angle = angle[:, None]
    c, s = angle.cos(), angle.sin()
    a, b = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def plain_append(st):
    _, _, kv, dn, dr = CACHES[st["case"]["kind"]]
    x, cache, slots = st["new_kv"], st["cache"], st["slots"].long()
    if st["case"]["kind"] in ("mla", "gla"):
        row = torch.cat([x[:, :kv * dn], turn(x[:, kv * dn:], st["pos"]).to(torch.bfloat16)], 1)
        cache.view(-1, kv * dn + dr)[slots] = row
        return cache
    k, v = turn(x[:, 0], st["pos"]), x[:, 1]
    page, at = slots // PAGE, slots % PAGE
    if st["case"]["kind"] == "gqa_fp8":
        bits = cache.view(torch.uint8)
        bits[page, 0, at] = (k / K_SCALE).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        bits[page, 1, at] = (v.float() / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return cache
    cache[page, 0, at], cache[page, 1, at] = k.to(torch.bfloat16), v
    return cache


def rows_of(st):
    """The cached rows of every sequence, one after the other."""
    start = st["kv_start"].long()
    t = torch.arange(st["total"], device=DEV)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = t - start[b]
    page = st["block_table"][b, pos // PAGE].long()
    return st["cache"].view(-1, st["cache"].shape[-1])[page * PAGE + pos % PAGE]


def plain_expand(st):
    c = st["case"]
    rows = rows_of(st)
    lat = rows[:, :c["groups"] * c["d_c"]].float().view(-1, c["groups"], c["d_c"]).transpose(0, 1)      # [G][T][d_c]
    lat = lat.repeat_interleave(c["heads"] // c["groups"], 0) if c["groups"] > 1 else lat.expand(c["heads"], -1, -1)
    k = torch.matmul(lat, st["w_uk"].float().transpose(1, 2)).to(torch.bfloat16)
    v = torch.matmul(lat, st["w_uv"].float()).to(torch.bfloat16)
    return dict(k=k, v=v, k_rope=rows[:, c["groups"] * c["d_c"]:].contiguous())


def plain_prefill(st):
    c = st["case"]
    H, KH = c["heads"], c["kv_heads"]
    out = torch.empty(st["q_nope"].shape[0], H, c["d_v"], dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(st["q_nope"].shape[0], H, dtype=torch.float32, device=DEV)
    q0 = k0 = 0
    for nq, nk in zip(st["q_lens"], st["k_lens"]):
        if nq:
            q = st["q_nope"][q0:q0 + nq].float().view(nq, KH, H // KH, -1).permute(1, 2, 0, 3).reshape(KH, -1, c["d_nope"])
            s = torch.matmul(q, st["k"][:, k0:k0 + nk].float().transpose(1, 2))
            if c["d_rope"]:
                qr = st["q_rope"][q0:q0 + nq].float().view(nq, KH, H // KH, -1).permute(1, 2, 0, 3).reshape(KH, -1, c["d_rope"])
                s += torch.matmul(qr, st["k_rope"][k0:k0 + nk].float().T)
            s = s.view(KH, H // KH, nq, nk).mul_(st["scale"])
            if c["causal"]:
                i, j = torch.arange(nq, device=DEV)[:, None], torch.arange(nk, device=DEV)
                s.masked_fill_(j > i + (nk - nq), -math.inf)
            m = s.amax(-1, keepdim=True)
            s.sub_(m).exp_()
            l = s.sum(-1, keepdim=True)
            o = torch.matmul(s.view(KH, -1, nk), st["v"][:, k0:k0 + nk].float()).view(KH, H // KH, nq, -1) / l
            out[q0:q0 + nq] = o.permute(2, 0, 1, 3).reshape(nq, H, -1).to(torch.bfloat16)
            lse[q0:q0 + nq] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(nq, H)
        q0, k0 = q0 + nq, k0 + nk
    return dict(out=out[:q0], lse=lse[:q0])


# ------------------------------------------------------- the work of one pass

def work(case):
    if case["op"] == "tables":
        cached, new = lengths(case, case["cached_lo"], case["cached_hi"], 1), lengths(case, case["new_lo"], case["new_hi"], 2)
        fresh = sum(pages_of(c + n) - pages_of(c) for c, n in zip(cached, new))
        # lengths in; lengths, starts, each new page twice, each token's position and slot out
        return {"bytes": 4 * (2 * case["batch"] + 3 * case["batch"] + 2 * fresh + 2 * sum(new)), "flops": 0}
    if case["op"] == "append":
        _, _, kv, dn, dr = CACHES[case["kind"]]
        row = kv * dn + dr if case["kind"] in ("mla", "gla") else 2 * kv * dn
        turned = dr if dr else kv * dn
        return {"bytes": case["tokens"] * (row * (2 + (1 if case["kind"] == "gqa_fp8" else 2)) + 8), "flops": 3 * turned * case["tokens"]}
    if case["op"] == "expand":
        T = sum(lengths(case, case["lo"], case["hi"], 3))
        H, G, dc, w = case["heads"], case["groups"], case["d_c"], case["d_k"] + case["d_v"]
        return {"bytes": 2 * (T * (G * dc + 64) + H * dc * w + T * H * w + T * 64), "flops": 2 * T * H * dc * w}
    q = lengths(case, case["q_lo"], case["q_hi"], 4)
    k = [a + b for a, b in zip(q, lengths(case, case["past_lo"], case["past_hi"], 5))]
    # the pairs that the mask leaves
    pairs = sum(nq * (nk - nq) + nq * (nq + 1) // 2 if case["causal"] else nq * nk for nq, nk in zip(q, k))
    dk = case["d_nope"] + case["d_rope"]
    return {"bytes": 2 * (sum(q) * case["heads"] * (dk + case["d_v"] + 2) + sum(k) * (case["kv_heads"] * (case["d_nope"] + case["d_v"]) + case["d_rope"])),
            "flops": 2 * pairs * case["heads"] * (dk + case["d_v"])}


# ------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None              # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "append":
        _, _, kv, dn, dr = CACHES[case["kind"]]
        cache, x = st["cache"].double(), st["new_kv"].double()
        width = dr if dr else dn
        head = x[:, kv * dn:] if dr else x[:, 0]
        # a pair as a complex number, turned by a unit one
        z = torch.view_as_complex(head.unflatten(-1, (width // 2, 2)).contiguous())
        rate = torch.exp(torch.arange(width // 2, device=DEV, dtype=torch.float64) * (-2 * math.log(ROPE_BASE) / width))
        unit = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), st["pos"].double()[:, None] * rate)
        head = torch.view_as_real(z * (unit if dr else unit[:, None])).flatten(-2)
        page, at = torch.div(st["slots"].long(), PAGE, rounding_mode="floor"), st["slots"].long() % PAGE
        if dr:
            cache[page, at] = torch.cat([x[:, :kv * dn], head], 1)
        else:
            scale = (K_SCALE, V_SCALE) if case["kind"] == "gqa_fp8" else (1.0, 1.0)
            cache[page, 0, at], cache[page, 1, at] = head / scale[0], x[:, 1] / scale[1]
        return cache
    if case["op"] == "expand":
        cols = case["groups"] * case["d_c"]
        table, flat = st["block_table"].cpu().tolist(), st["cache"].double()
        seqs = [flat[torch.tensor(table[b][:pages_of(n)], dtype=torch.int64, device=DEV)].flatten(0, 1)[:n] for b, n in enumerate(st["lens"])]
        rows = torch.cat(seqs)
        lat = rows[:, :cols].unflatten(1, (case["groups"], case["d_c"]))
        uk = st["w_uk"].double().unflatten(0, (case["groups"], -1))
        uv = st["w_uv"].double().unflatten(0, (case["groups"], -1))
        return dict(k=torch.einsum("tgc,ghdc->ghtd", lat, uk).flatten(0, 1), v=torch.einsum("tgc,ghcd->ghtd", lat, uv).flatten(0, 1), k_rope=rows[:, cols:])
    H, KH = case["heads"], case["kv_heads"]
    n = sum(st["q_lens"])
    out = torch.zeros(n, H, case["d_v"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(n, H, dtype=torch.float64, device=DEV)
    for h in range(H):
        q = st["q_nope"][:, h].double()
        k, v = st["k"][h // (H // KH)].double(), st["v"][h // (H // KH)].double()
        if case["d_rope"]:
            q, k = torch.cat([q, st["q_rope"][:, h].double()], 1), torch.cat([k, st["k_rope"].double()], 1)
        a = b = 0
        for nq, nk in zip(st["q_lens"], st["k_lens"]):
            if nq:
                s = st["scale"] * torch.einsum("id,jd->ij", q[a:a + nq], k[b:b + nk])
                if case["causal"]:
                    s = s + torch.full_like(s, -math.inf).triu(nk - nq + 1)
                lse[a:a + nq, h] = torch.logsumexp(s, 1)
                out[a:a + nq, h] = torch.softmax(s, 1) @ v[b:b + nk]
            a, b = a + nq, b + nk
    return dict(out=out, lse=lse)
