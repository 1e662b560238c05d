"""The prompt side on the GPU (kvattn_build_tables, kvattn_append_slots,
kvattn_expand_kv, kvattn_prefill) against the fp64 reference in
oracle/prompt.py.

Tolerances, from the arithmetic (a rounding to bf16 is off by at most 2^-8 of
the value, to e4m3 by 2^-4, in fp32 by 2^-24):
* tables: whole numbers, equal.
* append: copied parts equal; a turned pair is formed in double precision and
  rounded once, as the reference's is, so at most one bf16 step apart (a
  double's rounding next to a tie) and hardly ever; e4m3 likewise.
* expand: products of bf16 are exact in fp32, d_c <= 512 of them are added in
  fp32: 1e-5 of sum |c w| covers the sums (512 * 2^-24 = 3e-5 if every rounding
  went one way; they do not over more than a third), and one rounding: 2^-8 |y|.
* prefill: a score is a sum of at most 192 exact products in fp32, off by at
  most 192 * 2^-24 = 1.2e-5 of scale * sum |q k| (`reach`), and the exponent's
  fma, 2^x (2 ulp) and the sums add less than 1e-5 + 2^-23 |m| with |m| <= reach;
  delta = 1.5e-5 * reach + 1e-5.  A weight is off by 2 delta (itself and the
  denominator) and rounded to bf16 for P.V: |out| off by (2^-8 + 2 delta) sum p
  |v|, and its own rounding 2^-8 |out| when it is stored in bf16.  lse is off by
  delta + 2^-22 |lse|.
"""

import numpy as np
import pytest

from oracle import prompt
from shared_kv_caches_b200 import kvattn as K
from shared_kv_caches_b200 import workloads as W

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from shared_kv_caches_b200 import build
    build.build()
    return torch.device("cuda:0")


def bits(rng, *shape, scale=1.0):
    return W.f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def f64(b):
    return W.bf16_bits_to_f32(np.asarray(b)).astype(np.float64)


def up(b, dev):
    from shared_kv_caches_b200.device import bf16_tensor
    return bf16_tensor(b, dev)


def i32(x, dev):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def down(t):
    return t.detach().double().cpu().numpy()


def word(dev):
    import torch
    return torch.zeros(1, dtype=torch.int32, device=dev)


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


# ------------------------------------------------------------------ tables

def table_case(rng, cached, new, mpps=None, spare=3, shrink=0):
    cached, new = np.asarray(cached), np.asarray(new)
    held = -(-np.maximum(cached, 0) // 64)
    need = -(-np.maximum(cached + new, 0) // 64)
    mpps = int(max(need.max(), 1)) if mpps is None else mpps
    num_pages = int(need.sum()) + spare
    perm = rng.permutation(num_pages)
    table = np.full((len(cached), mpps), -7, dtype=np.int64)
    at = 0
    for b, h in enumerate(held):
        table[b, :min(h, mpps)] = perm[at:at + min(h, mpps)]
        at += h
    free = perm[at:]
    count = max(len(free) - shrink, 0)
    return table, np.concatenate([free, np.full(at, -1)])[:num_pages], count, num_pages


def run_tables(dev, cached, new, table, free, count, max_tokens, **kw):
    err = word(dev)
    r = K.build_tables_tensors(i32(cached, dev), i32(new, dev), i32(free, dev), i32([count], dev), i32(table, dev),
                               max_tokens, device_error=err, **kw)
    return {k: v.cpu().numpy().astype(np.int64) for k, v in r.items()} | {"err": int(err.item())}


def same_tables(got, ref):
    for k in ref:
        np.testing.assert_array_equal(got[k], ref[k], err_msg=k)


@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([0], [0]), ([5], [200]), ([1, 0, 64, 63, 128], [1, 1, 1, 1, 1]),
    ([0, 10, 0, 64], [0, 0, 130, 64]), ([0] * 40, list(range(40))),
])
def test_tables_small(dev, cached, new):
    rng = np.random.default_rng(1)
    table, free, count, pages = table_case(rng, cached, new)
    m = sum(new) + 5
    same_tables(run_tables(dev, cached, new, table, free, count, m),
                prompt.build_tables(cached, new, free, count, table, m, pages))


@pytest.mark.parametrize("batch,hi,past", [(1, 40000, 0), (7, 9000, 3000), (1025, 3, 700), (3000, 64, 0), (16384, 1, 129)])
def test_tables_large(dev, batch, hi, past):
    rng = np.random.default_rng(batch)
    cached, new = rng.integers(0, past + 1, batch), rng.integers(0, hi + 1, batch)
    table, free, count, pages = table_case(rng, cached, new)
    m = int(new.sum())
    same_tables(run_tables(dev, cached, new, table, free, count, m),
                prompt.build_tables(cached, new, free, count, table, m, pages))


@pytest.mark.parametrize("shrink", [1, 4, 100])
def test_tables_pool_runs_out(dev, shrink):
    rng = np.random.default_rng(shrink)
    cached, new = rng.integers(0, 200, 30), rng.integers(0, 300, 30)
    table, free, count, pages = table_case(rng, cached, new, shrink=shrink, spare=0)
    m = int(new.sum()) + 3
    ref = prompt.build_tables(cached, new, free, count, table, m, pages)
    assert ref["err"] == prompt.ERR_POOL
    same_tables(run_tables(dev, cached, new, table, free, count, m), ref)


@pytest.mark.parametrize("case", ["tokens", "long", "negative", "bad_free", "bad_held", "no_free", "count"])
def test_tables_bad_requests_get_nothing(dev, case):
    rng = np.random.default_rng(5)
    cached, new = np.array([10, 64, 0, 130, 7]), np.array([3, 100, 64, 0, 70])
    table, free, count, pages = table_case(rng, cached, new)
    m, want = int(new.sum()), {"tokens": prompt.ERR_TOKENS, "long": prompt.ERR_LONG, "negative": prompt.ERR_LENGTH,
                               "bad_free": prompt.ERR_PAGE, "bad_held": prompt.ERR_PAGE, "no_free": prompt.ERR_POOL,
                               "count": prompt.ERR_LENGTH}[case]
    if case == "tokens":
        m = 150
    elif case == "long":
        cached[1] = 64 * table.shape[1]
    elif case == "negative":
        new[1], cached[3] = -5, -1
    elif case == "bad_free":
        free[count - 2] = pages
    elif case == "bad_held":
        table[0, 0] = -1
    elif case == "no_free":
        count = 0
    else:
        count = pages + 9
        free[:] = rng.permutation(pages)
    ref = prompt.build_tables(cached, new, free, count, table, m, pages)
    assert ref["err"] == want
    same_tables(run_tables(dev, cached, new, table, free, count, m), ref)


def test_tables_in_place_step_replays_in_a_graph(dev):
    """Lengths and free list updated in place: each replay is one more step."""
    import torch
    cached, new = np.array([62, 0, 127]), np.array([1, 1, 2])
    rng = np.random.default_rng(8)
    table, free, count, pages = table_case(rng, cached, new + 20, mpps=8)
    lens, cnt, tab, one, pool = i32(cached, dev), i32([count], dev), i32(table, dev), i32(new, dev), i32(free, dev)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        r = K.build_tables_tensors(lens, one, pool, cnt, tab, 6, inplace=True)
    ref_c, ref_t, ref_n = cached, table, count
    for _ in range(6):
        g.replay()
        torch.cuda.synchronize()
        ref = prompt.build_tables(ref_c, new, free, ref_n, ref_t, 6, pages)
        ref.pop("err")
        same_tables({k: v.cpu().numpy() for k, v in r.items()}, ref)
        ref_c, ref_t, ref_n = ref["seq_lens"], ref["block_table"], int(ref["free_left"][0])


# ------------------------------------------------------------------ append

def turned_close(got, ref, step):
    """Equal but for values next to a tie, which may land one step away."""
    off = np.abs(got - ref) > 0
    assert np.all(np.abs(got - ref)[off] <= 2 * step * np.abs(ref)[off] + 2.0 ** -130)
    assert off.mean() < 1e-3


def bf16_round(x):
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


@pytest.mark.parametrize("variant,heads,kv,dn,dr", [("mla", 128, 1, 512, 64), ("gla", 8, 4, 128, 32), ("mlra", 4, 2, 64, 16),
                                                    ("mla", 4, 1, 72, 0), ("mla", 4, 1, 64, 128)])
@pytest.mark.parametrize("base", [0.0, W.ROPE_BASE])
def test_append_latent_rows(dev, variant, heads, kv, dn, dr, base):
    import torch
    rng = np.random.default_rng(3)
    row, pages, n = kv * dn + dr, 9, 203
    cache, rows = bits(rng, pages, 64, row), bits(rng, n, row)
    slots = rng.permutation(pages * 64)[:n].astype(np.int32)
    slots[[0, 50]] = -1
    pos = rng.integers(0, 1 << 20, n)
    pos[3], pos[4] = 0, -5
    p = K.make_params(1, heads, kv, dn, dr, pages, pages, 0)
    t, err = up(cache, dev), word(dev)
    K.append_slots_tensor(K.VARIANTS[variant], p, up(rows, dev), i32(pos, dev), i32(slots, dev), t, base, err)
    ref = prompt.append_rows(f64(cache), f64(rows), pos, slots, [(kv * dn, dr)] if dr else [], base)
    got = down(t)
    assert int(err.item()) == 0
    np.testing.assert_array_equal(got[..., :kv * dn], ref[..., :kv * dn])
    if base and dr:
        turned_close(got[..., kv * dn:], bf16_round(ref[..., kv * dn:]), BF16)
    else:
        np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("variant,kv,d", [("gqa", 8, 128), ("gqa", 2, 64), ("mqa", 1, 256), ("gqa", 3, 512), ("gta", 4, 128)])
def test_append_head_rows(dev, variant, kv, d):
    rng = np.random.default_rng(4)
    planes, base = (1, 0.0) if variant == "gta" else (2, W.ROPE_BASE)
    pages, n = 5, 150
    cache, rows = bits(rng, pages, planes, 64, kv * d), bits(rng, n, planes, kv * d)
    slots, pos = rng.permutation(pages * 64)[:n], rng.integers(0, 40000, n)
    p = K.make_params(1, 2 * kv, kv, d, 0, pages, pages, 0)
    t = up(cache, dev)
    K.append_slots_tensor(K.VARIANTS[variant], p, up(rows, dev), i32(pos, dev), i32(slots, dev), t, base)
    got = down(t)
    for pl in range(planes):
        turn = base if pl == 0 else 0.0
        ref = prompt.append_rows(f64(cache[:, pl]), f64(rows[:, pl]), pos, slots, [(h * d, d) for h in range(kv)], turn)
        if turn:
            turned_close(got[:, pl], bf16_round(ref), BF16)
        else:
            np.testing.assert_array_equal(got[:, pl], ref)


@pytest.mark.parametrize("base", [0.0, W.ROPE_BASE])
def test_append_quantises_into_the_fp8_cache(dev, base):
    import torch
    from oracle import oracle
    rng = np.random.default_rng(6)
    kv, d, pages, n = 8, 128, 4, 130
    cache = rng.integers(0, 256, (pages, 2, 64, kv, d)).astype(np.uint8)
    rows = bits(rng, n, 2, kv * d, scale=3.0)
    rows[5, 1, :4] = W.f32_to_bf16_bits(np.array([1e5, -1e5, 0.0, 2.0 ** -12], np.float32))
    rows[6, 1, 0] = W.BF16_NAN
    slots, pos = rng.permutation(pages * 64)[:n], rng.integers(0, 40000, n)
    p = K.make_params(1, 32, kv, d, 0, pages, pages, 0, cache_dtype=K.KVATTN_CACHE_FP8_E4M3, k_scale=0.37, v_scale=1.7)
    t = torch.from_numpy(cache).to(dev)
    K.append_slots_tensor(K.KVATTN_GQA, p, up(rows, dev), i32(pos, dev), i32(slots, dev), t, base)
    got = t.cpu().numpy()
    ks, vs = float(np.float32(0.37)), float(np.float32(1.7))
    flat = got.transpose(0, 2, 1, 3, 4).reshape(pages * 64, 2, kv * d)
    old = cache.transpose(0, 2, 1, 3, 4).reshape(pages * 64, 2, kv * d)
    rest = np.setdiff1d(np.arange(pages * 64), slots)
    np.testing.assert_array_equal(flat[rest], old[rest])
    k = prompt.append_rows(np.zeros((pages, 64, kv * d)), f64(rows[:, 0]), pos, slots, [(h * d, d) for h in range(kv)], base)
    k = k.reshape(pages * 64, kv * d)[slots] / ks
    v = (f64(rows[:, 1]).astype(np.float32) / np.float32(vs)).astype(np.float64)
    for have, want in ((flat[slots, 0], k), (flat[slots, 1], v)):
        code = W.f32_to_e4m3_bits(want)
        # next to a tie the two may round apart: neighbouring codes
        apart = np.abs(have.astype(int) - code.astype(int))
        assert apart.max() <= 1 and (apart > 0).mean() < 1e-3
    assert oracle.e4m3_value(flat[slots[5], 1, 0]) == 448.0 and flat[slots[6], 1, 0] & 0x7F == 0x7F


def test_append_bad_slots_are_skipped(dev):
    rng = np.random.default_rng(7)
    cache, rows = bits(rng, 2, 64, 72), bits(rng, 4, 72)
    p = K.make_params(1, 4, 1, 64, 8, 2, 2, 0)
    t, err = up(cache, dev), word(dev)
    K.append_slots_tensor(K.KVATTN_MLA, p, up(rows, dev), i32([1, 2, 3, 4], dev), i32([128, -2, 5, -1], dev), t, 0.0, err)
    ref = f64(cache)
    ref[0, 5] = f64(rows[2])
    np.testing.assert_array_equal(down(t), ref)
    assert int(err.item()) == K.KVATTN_DEVERR_PAGE_OUT_OF_RANGE


# ------------------------------------------------------------------ expand

def expand_case(rng, dev, H, G, dc, dr, dk, dv, lens, paged=True, extra=0):
    need = [-(-n // 64) for n in lens]
    mpps = max(need + [1])
    pages = (sum(need) + 2) if paged else mpps * len(lens)
    cache = bits(rng, pages, 64, G * dc + dr)
    if paged:
        perm, at = rng.permutation(pages), 0
        table = np.full((len(lens), mpps), pages + 5, dtype=np.int32)
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
    else:
        table = None
    for b, n in enumerate(lens):       # slots past the length hold anything
        if n % 64:
            pg = table[b, n // 64] if paged else b * mpps + n // 64
            cache[pg, n % 64:] = W.BF16_NAN
    uk, uv = bits(rng, H, dk, dc, scale=dc ** -0.5), bits(rng, H, dc, dv, scale=dc ** -0.5)
    p = K.make_params(len(lens), H, G, dc, dr, mpps, pages, 0)
    return cache, table, uk, uv, p, mpps


def check_expand(got, cache, table, uk, uv, groups, lens, mpps):
    st = starts(lens)
    for b, n in enumerate(lens):
        rows = prompt.gather(f64(cache), table, b, n, mpps)
        k, v, ka, va = prompt.expand(rows, f64(uk), f64(uv), groups)
        gk, gv = down(got["k"][:, st[b]:st[b + 1]]), down(got["v"][:, st[b]:st[b + 1]])
        assert np.all(np.abs(gk - k) <= BF16 * np.abs(k) + 1e-5 * ka)
        assert np.all(np.abs(gv - v) <= BF16 * np.abs(v) + 1e-5 * va)
        if got["k_rope"] is not None:
            np.testing.assert_array_equal(down(got["k_rope"][st[b]:st[b + 1]]), rows[:, groups * uk.shape[2]:])


@pytest.mark.parametrize("H,G,dc,dr,dk,dv,lens,paged", [
    (4, 1, 512, 64, 128, 128, [1, 0, 63, 64, 65, 127, 128, 129, 300], True),
    (8, 2, 256, 64, 128, 128, [200, 1], True),
    (6, 2, 128, 32, 64, 128, [130, 0, 70], True),
    (2, 1, 128, 16, 64, 64, [64] * 33, True),
    (4, 2, 64, 64, 128, 128, [2000, 1, 500], True),
    (3, 1, 64, 16, 40, 72, [100, 129], False),
    (2, 1, 64, 0, 8, 8, [257], True),
    (130, 1, 64, 64, 128, 64, [64, 64], True),
])
def test_expand_matches_reference(dev, H, G, dc, dr, dk, dv, lens, paged):
    rng = np.random.default_rng(H + dc)
    cache, table, uk, uv, p, mpps = expand_case(rng, dev, H, G, dc, dr, dk, dv, lens, paged)
    err = word(dev)
    got = K.expand_kv_tensors(K.KVATTN_MLA if G == 1 else K.KVATTN_GLA, p, up(cache, dev),
                              None if table is None else i32(table, dev), i32(starts(lens), dev), up(uk, dev), up(uv, dev),
                              sum(lens), err)
    assert int(err.item()) == 0
    check_expand(got, cache, table, uk, uv, G, lens, mpps)


@pytest.mark.parametrize("H,R,dc,dk,dv", [(6, 4, 128, 128, 128), (3, 2, 64, 64, 40)])
def test_expand_branches(dev, H, R, dc, dk, dv):
    """MLRA: every head's keys and values of each branch, weights' blocks side by side and stacked."""
    rng = np.random.default_rng(R)
    lens = [130, 0, 65]
    cache, table, _, _, p, mpps = expand_case(rng, dev, H, R, dc, 32, dk, dv, lens)
    uk, uv = bits(rng, H, dk, R * dc, scale=dc ** -0.5), bits(rng, H, R * dc, dv, scale=dc ** -0.5)
    got = K.expand_kv_tensors(K.KVATTN_MLRA, p, up(cache, dev), i32(table, dev), i32(starts(lens), dev), up(uk, dev), up(uv, dev),
                              sum(lens))
    assert got["k"].shape == (H * R, sum(lens), dk)
    for r in range(R):
        cols = np.r_[r * dc:(r + 1) * dc, R * dc:R * dc + 32]
        one = dict(k=got["k"][r::R], v=got["v"][r::R], k_rope=got["k_rope"])
        check_expand(one, cache[..., cols], table, uk[..., r * dc:(r + 1) * dc], uv[:, r * dc:(r + 1) * dc], 1, lens, mpps)


def test_expand_leaves_rows_past_the_last_sequence(dev):
    import torch
    rng = np.random.default_rng(2)
    lens = [70, 130]
    cache, table, uk, uv, p, mpps = expand_case(rng, dev, 2, 1, 64, 16, 64, 128, lens)
    n = sum(lens) + 77
    k = torch.full((2, n, 64), 7.0, dtype=torch.bfloat16, device=dev)
    v = torch.full((2, n, 128), 7.0, dtype=torch.bfloat16, device=dev)
    kr = torch.full((n, 16), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(K.kvattn_expand_workspace_size(K.KVATTN_MLA, p, n), dtype=torch.uint8, device=dev)
    c, t, s, a, b = up(cache, dev), i32(table, dev), i32(starts(lens), dev), up(uk, dev), up(uv, dev)
    assert K.kvattn_expand_kv(K.KVATTN_MLA, p, c.data_ptr(), t.data_ptr(), s.data_ptr(), n, 64, 128, a.data_ptr(),
                              b.data_ptr(), k.data_ptr(), v.data_ptr(), kr.data_ptr(), ws.data_ptr(), ws.numel(), None,
                              torch.cuda.current_stream().cuda_stream) == 0
    check_expand(dict(k=k, v=v, k_rope=kr), cache, table, uk, uv, 1, lens, mpps)
    for x in (k[:, sum(lens):], v[:, sum(lens):], kr[sum(lens):]):
        assert bool((x == 7.0).all())


def test_expand_bad_page_gives_zeros_and_the_bit(dev):
    rng = np.random.default_rng(9)
    lens = [100, 200]
    cache, table, uk, uv, p, mpps = expand_case(rng, dev, 3, 1, 64, 16, 64, 64, lens)
    table[1, 2] = -3
    err = word(dev)
    got = K.expand_kv_tensors(K.KVATTN_MLA, p, up(cache, dev), i32(table, dev), i32(starts(lens), dev), up(uk, dev),
                              up(uv, dev), sum(lens), err)
    assert int(err.item()) == K.KVATTN_DEVERR_PAGE_OUT_OF_RANGE
    for x in (got["k"][:, 228:292], got["v"][:, 228:292], got["k_rope"][228:292]):
        assert bool((x == 0).all())
    check_expand({k: v[..., :228, :] for k, v in got.items()}, cache, table, uk, uv, 1, [100, 128], mpps)


# ----------------------------------------------------------------- prefill

def prefill_case(rng, H, KH, dn, dr, dv, ql, kl, slack=9):
    tq, tk = sum(ql) + slack, sum(kl) + slack
    x = dict(q=bits(rng, tq, H, dn), k=bits(rng, KH, tk, dn), v=bits(rng, KH, tk, dv),
             qr=bits(rng, tq, H, dr) if dr else None, kr=bits(rng, tk, dr) if dr else None)
    for name in ("k", "v"):
        x[name][:, sum(kl):] = W.BF16_NAN
    if dr:
        x["kr"][sum(kl):] = W.BF16_NAN
    x["q"][sum(ql):] = W.BF16_NAN
    return x


def check_prefill(got, x, ql, kl, scale, causal, fp32=False, skip=()):
    H, KH = x["q"].shape[1], x["k"].shape[0]
    out, lse = down(got["out"]), down(got["lse"])
    qs, ks = starts(ql), starts(kl)
    for b in range(len(ql)):
        if b in skip:
            continue
        a, e, c, d = qs[b], qs[b + 1], ks[b], ks[b + 1]
        for h in range(H):
            q, k = f64(x["q"][a:e, h]), f64(x["k"][h // (H // KH), c:d])
            if x["qr"] is not None:
                q = np.concatenate([q, f64(x["qr"][a:e, h])], 1)
                k = np.concatenate([k, f64(x["kr"][c:d])], 1)
            ro, rl, mass, reach = prompt.attention(q, k, f64(x["v"][h // (H // KH), c:d]), scale, causal)
            delta = 1.5e-5 * reach + 1e-5
            tol = (BF16 + 2 * delta)[:, None] * mass + (0 if fp32 else BF16) * np.abs(ro) + 1e-30
            assert np.all(np.abs(out[a:e, h] - ro) <= tol), (b, h, np.abs(out[a:e, h] - ro).max())
            none = np.isinf(rl)
            np.testing.assert_array_equal(lse[a:e, h][none], rl[none])
            assert np.all(np.abs(lse[a:e, h][~none] - rl[~none]) <= delta[~none] + 2.0 ** -22 * np.abs(rl[~none])), (b, h)


def call(dev, x, ql, kl, scale, causal, **kw):
    t = {k: None if v is None else up(v, dev) for k, v in x.items()}
    return K.prefill_tensors(t["q"], t["qr"], t["k"], t["kr"], t["v"], i32(starts(ql), dev), i32(starts(kl), dev), scale,
                             causal=causal, **kw)


LENS = [([1], [1]), ([1], [200]), ([127], [127]), ([128], [128]), ([129], [129]), ([256], [256]), ([257], [300]),
        ([0, 3, 0, 130, 1], [5, 3, 0, 400, 64]), ([300, 2], [300, 1000]), ([2, 200], [0, 150])]


@pytest.mark.parametrize("ql,kl", LENS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("slack", [9, 5000])
def test_prefill_lengths(dev, ql, kl, causal, slack):
    """Lengths around the tiles, cached prefixes, sequences without queries or keys, rows whose mask leaves nothing.
    With little room for rows every CTA lists the tiles, with much the plan kernel does."""
    rng = np.random.default_rng(sum(ql) + sum(kl))
    x = prefill_case(rng, 2, 2, 128, 64, 128, ql, kl, slack)
    err = word(dev)
    got = call(dev, x, ql, kl, 192 ** -0.5, causal, device_error=err)
    assert int(err.item()) == 0
    check_prefill(got, x, ql, kl, 192 ** -0.5, causal)


@pytest.mark.parametrize("H,KH,dn,dr,dv", [(4, 1, 128, 0, 128), (8, 2, 64, 0, 64), (3, 3, 64, 16, 64), (2, 1, 64, 64, 128),
                                           (2, 2, 128, 64, 64), (2, 2, 72, 8, 40), (9, 3, 8, 0, 8), (2, 2, 128, 32, 96),
                                           (17, 17, 64, 0, 128)])
@pytest.mark.parametrize("fp32", [False, True])
def test_prefill_head_layouts(dev, H, KH, dn, dr, dv, fp32):
    rng = np.random.default_rng(H * dn + dv)
    ql, kl = [150, 1, 77], [150, 140, 300]
    x = prefill_case(rng, H, KH, dn, dr, dv, ql, kl)
    got = call(dev, x, ql, kl, (dn + dr) ** -0.5, True, out_fp32=fp32)
    check_prefill(got, x, ql, kl, (dn + dr) ** -0.5, True, fp32)


def test_prefill_heads_that_share_q_nope(dev):
    rng = np.random.default_rng(22)
    ql, kl = [140, 20], [140, 300]
    x = prefill_case(rng, 12, 12, 128, 64, 128, ql, kl)
    q = x["q"][:, :3].copy()
    x["q"] = np.repeat(q, 4, axis=1)
    t = {k: up(v, dev) for k, v in x.items()}
    got = K.prefill_tensors(up(q, dev), t["qr"], t["k"], t["kr"], t["v"], i32(starts(ql), dev), i32(starts(kl), dev), 0.08)
    check_prefill(got, x, ql, kl, 0.08, True)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.0])
def test_prefill_scales(dev, scale):
    """A negative scale, none (every key weighs the same), and scores far apart."""
    rng = np.random.default_rng(11)
    ql, kl = [140], [270]
    x = prefill_case(rng, 2, 2, 128, 64, 128, ql, kl)
    check_prefill(call(dev, x, ql, kl, scale, True), x, ql, kl, scale, True)


def test_prefill_rising_maxima(dev):
    """Scores that keep growing along the keys: the running maximum moves and outputs are rescaled in every tile."""
    rng = np.random.default_rng(12)
    ql, kl = [130], [900]
    x = prefill_case(rng, 1, 1, 64, 0, 64, ql, kl)
    ramp = np.linspace(0.0, 4.0, 900)[:, None]
    x["k"][0, :900] = W.f32_to_bf16_bits((f64(x["k"][0, :900]) * 0.1 + ramp).astype(np.float32))
    x["q"][:130, 0] = W.f32_to_bf16_bits((np.abs(f64(x["q"][:130, 0])) + 0.2).astype(np.float32))
    check_prefill(call(dev, x, ql, kl, 0.5, False), x, ql, kl, 0.5, False)


def test_prefill_strided_views(dev):
    """Keys and values token by token, queries as slices of one projection, output into a wider tensor."""
    import torch
    rng = np.random.default_rng(13)
    H, KH, dn, dr, dv, ql, kl = 4, 2, 64, 16, 72, [100, 33], [100, 160]
    x = prefill_case(rng, H, KH, dn, dr, dv, ql, kl, slack=0)
    tq, tk = sum(ql), sum(kl)
    qq = torch.zeros(tq, H, 96, dtype=torch.bfloat16, device=dev)
    qq[..., :dn], qq[..., 72:72 + dr] = up(x["q"], dev), up(x["qr"], dev)
    kv = torch.zeros(tk, KH, dn + dv, dtype=torch.bfloat16, device=dev)
    kv[..., :dn], kv[..., dn:] = up(x["k"], dev).transpose(0, 1), up(x["v"], dev).transpose(0, 1)
    row = torch.zeros(tk, 40, dtype=torch.bfloat16, device=dev)
    row[:, 24:] = up(x["kr"], dev)
    wide = torch.full((tq, H + 1, 80), 3.0, dtype=torch.bfloat16, device=dev)
    kv_t = kv.transpose(0, 1)
    got = K.prefill_tensors(qq[..., :dn], qq[..., 72:72 + dr], kv_t[..., :dn], row[:, 24:], kv_t[..., dn:],
                            i32(starts(ql), dev), i32(starts(kl), dev), 0.1, out=wide[:, :H, :dv])
    check_prefill(got, x, ql, kl, 0.1, True)
    assert bool((wide[:, H] == 3.0).all()) and bool((wide[..., dv:] == 3.0).all())


def test_prefill_one_head_one_token_and_broadcast_axes(dev):
    """Axes of one element may have any stride; a broadcast axis is refused."""
    import torch
    rng = np.random.default_rng(21)
    x = prefill_case(rng, 1, 1, 64, 0, 64, [1], [1], slack=0)
    t = {k: None if v is None else up(v, dev) for k, v in x.items()}
    q = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device=dev)
    q[:, 1:2] = t["q"]
    got = K.prefill_tensors(q[:, 1:2].as_strided((1, 1, 64), (7, 3, 1), 64), None, t["k"], None, t["v"], i32([0, 1], dev),
                            i32([0, 1], dev), 0.1)
    check_prefill(got, x, [1], [1], 0.1, True)
    with pytest.raises(ValueError):
        K.prefill_tensors(t["q"].expand(1, 4, 64), None, t["k"].expand(4, 1, 64), None, t["v"].expand(4, 1, 64),
                          i32([0, 1], dev), i32([0, 1], dev), 0.1)


def test_prefill_without_keys(dev):
    """No key rows at all: zeros and -inf for every query."""
    import torch
    z = torch.zeros(2, 0, 64, dtype=torch.bfloat16, device=dev)
    got = K.prefill_tensors(torch.ones(200, 2, 64, dtype=torch.bfloat16, device=dev), None, z, None, z, i32([0, 150, 200], dev),
                            i32([0, 0, 0], dev), 0.1)
    assert bool((got["out"] == 0).all()) and bool(torch.isinf(got["lse"]).all())


def test_prefill_leaves_rows_past_the_last_sequence(dev):
    import torch
    rng = np.random.default_rng(14)
    ql, kl = [130, 5], [130, 9]
    x = prefill_case(rng, 2, 2, 64, 0, 64, ql, kl, slack=300)
    out = torch.full((435, 2, 64), 9.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((435, 2), 9.0, dtype=torch.float32, device=dev)
    got = call(dev, x, ql, kl, 0.1, True, out=out, lse=lse)
    check_prefill(got, x, ql, kl, 0.1, True)
    assert bool((out[135:] == 9.0).all()) and bool((lse[135:] == 9.0).all())


def test_prefill_nothing_passes_between_sequences(dev):
    """A sequence whose keys and values are NaN or infinite spoils only itself."""
    rng = np.random.default_rng(15)
    ql, kl = [60, 70, 80], [60, 70, 200]
    x = prefill_case(rng, 2, 2, 128, 64, 128, ql, kl)
    x["k"][:, 60:130], x["v"][:, 60:100], x["v"][:, 100:130] = W.BF16_NAN, W.BF16_NAN, 0x7F80
    x["q"][60:130] = W.BF16_NAN
    for causal in (True, False):
        check_prefill(call(dev, x, ql, kl, 0.1, causal), x, ql, kl, 0.1, causal, skip=(1,))


@pytest.mark.parametrize("ql,kl,at", [([200], [200], [0, 95, 96, 128, 150, 199]), ([300], [430], [130, 131, 300, 429]),
                                      ([70, 260], [70, 500], [69, 100, 309, 333, 569]), ([40], [20], [0, 19]),
                                      ([257], [257], [255, 256]), ([96], [1000], [900, 904, 905, 999])])
@pytest.mark.parametrize("fp32", [False, True])
def test_prefill_values_that_are_not_finite(dev, ql, kl, at, fp32):
    """A token whose value is NaN or infinite reaches the queries that attend it, in the columns that are, and no other."""
    rng = np.random.default_rng(26)
    x = prefill_case(rng, 3, 3, 128, 64, 128, ql, kl)
    clean = {k: None if v is None else v.copy() for k, v in x.items()}
    inf, ninf = 0x7F80, 0xFF80
    for i, t in enumerate(at):
        x["v"][i % 3, t, 5 * i:5 * i + 2] = W.BF16_NAN
        x["v"][1, t, 70 + i], x["v"][2, t, 127 - i] = inf, ninf
    x["k"][0, at[-1], 3] = W.BF16_NAN                       # a key: its queries' whole rows
    for causal in (True, False):
        got = call(dev, x, ql, kl, 0.07, causal, out_fp32=fp32)
        ref = call(dev, clean, ql, kl, 0.07, causal, out_fp32=fp32)
        out, lse, want, want_lse = (down(got["out"]), down(got["lse"]), down(ref["out"]), down(ref["lse"]))
        qs, ks = starts(ql), starts(kl)
        for b in range(len(ql)):
            nq, nk = ql[b], kl[b]
            for h in range(3):
                v = f64(x["v"][h, ks[b]:ks[b + 1]])
                for i in range(nq):
                    n = min(nk, max(i + nk - nq + 1, 0)) if causal else nk
                    row, line = out[qs[b] + i, h], want[qs[b] + i, h]
                    if h == 0 and ks[b] <= at[-1] < ks[b] + n:
                        assert np.isnan(row).all() and np.isnan(lse[qs[b] + i, h])
                        continue
                    with np.errstate(invalid="ignore"):
                        add = np.where(np.isfinite(v[:n]), 0.0, v[:n]).sum(0) if n else np.zeros(128)
                    np.testing.assert_array_equal(np.isnan(row), np.isnan(add))
                    np.testing.assert_array_equal(row[np.isinf(add)], add[np.isinf(add)])
                    fine = np.isfinite(add)
                    # the other columns lose or gain nothing
                    np.testing.assert_array_equal(row[fine], line[fine])
                    assert lse[qs[b] + i, h] == want_lse[qs[b] + i, h]


def test_prefill_bad_starts_set_the_bit(dev):
    import torch
    rng = np.random.default_rng(16)
    x = prefill_case(rng, 1, 1, 64, 0, 64, [50, 60, 70], [50, 60, 70])
    t = {k: None if v is None else up(v, dev) for k, v in x.items()}
    for room in (0, 5000):
        t["q"] = torch.cat([t["q"], torch.zeros(room, 1, 64, dtype=torch.bfloat16, device=dev)])
        far = 6000
        for q, k in (([0, 50, 110, far], [0, 50, 110, 180]), ([0, 50, 110, 180], [0, 50, 110, far]),
                     ([0, 50, 110, 90], [0, 50, 110, 180]), ([0, 50, 110, 180], [0, 50, 110, 90])):
            check_bad_starts(dev, x, t, q, k)


def check_bad_starts(dev, x, t, q, k):
    err = word(dev)
    got = K.prefill_tensors(t["q"], None, t["k"], None, t["v"], i32(q, dev), i32(k, dev), 0.1, device_error=err)
    assert int(err.item()) == K.KVATTN_DEVERR_BAD_LENGTH
    check_prefill(got, x, [50, 60], [50, 60], 0.1, True)


def test_prefill_many_sequences(dev):
    """More sequences than a block of the plan has threads, most of them short."""
    rng = np.random.default_rng(17)
    ql = rng.integers(0, 4, 1500).tolist()
    kl = [a + int(b) for a, b in zip(ql, rng.integers(0, 3, 1500))]
    x = prefill_case(rng, 1, 1, 64, 0, 64, ql, kl)
    check_prefill(call(dev, x, ql, kl, 0.1, True), x, ql, kl, 0.1, True)


def test_prefill_more_items_than_sms(dev):
    """Several items a CTA: query tiles, rings and TMEM are taken over from item to item."""
    rng = np.random.default_rng(18)
    ql, kl = [700, 3, 390], [700, 260, 520]
    x = prefill_case(rng, 41, 41, 64, 0, 64, ql, kl)
    check_prefill(call(dev, x, ql, kl, 0.125, True), x, ql, kl, 0.125, True)


def test_prefill_twice_is_the_same_and_streams_do_not_meet(dev):
    """Two calls at once on two streams, each with its own workspace, and a captured call replayed."""
    import torch
    rng = np.random.default_rng(19)
    ql, kl = [400, 100], [600, 100]
    x = prefill_case(rng, 8, 8, 128, 64, 128, ql, kl)
    t = {k: up(v, dev) for k, v in x.items()}
    qs, ks = i32(starts(ql), dev), i32(starts(kl), dev)
    torch.cuda.synchronize()

    def go():
        return K.prefill_tensors(t["q"], t["qr"], t["k"], t["kr"], t["v"], qs, ks, 0.07)["out"][:sum(ql)]
    one, side = go(), [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for s in side:
            with torch.cuda.stream(s):
                got.append(go())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kept = go()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for y in got + [kept]:
        assert torch.equal(one, y)


def test_prefill_and_expand_of_the_largest_batch(dev):
    """16384 sequences of no or one token."""
    rng = np.random.default_rng(23)
    ql = rng.integers(0, 2, 16384).tolist()
    x = prefill_case(rng, 1, 1, 8, 0, 8, ql, ql)
    err = word(dev)
    got = call(dev, x, ql, ql, 0.1, True, device_error=err)
    assert int(err.item()) == 0
    n = sum(ql)
    # one key each: the output is its value, lse the score
    np.testing.assert_array_equal(down(got["out"])[:n, 0], f64(x["v"][0, :n]))
    s = 0.1 * (f64(x["q"][:n, 0]) * f64(x["k"][0, :n])).sum(1)
    assert np.abs(down(got["lse"])[:n, 0] - s).max() <= 1e-5
    cache, table, uk, uv, p, mpps = expand_case(rng, dev, 2, 1, 64, 8, 8, 8, ql)
    e = K.expand_kv_tensors(K.KVATTN_MLA, p, up(cache, dev), i32(table, dev), i32(starts(ql), dev), up(uk, dev), up(uv, dev), n, err)
    assert int(err.item()) == 0
    rows = np.array([f64(cache[table[b, 0], 0]) for b in range(16384) if ql[b]])
    k, v, ka, va = prompt.expand(rows, f64(uk), f64(uv), 1)
    assert np.all(np.abs(down(e["k"]) - k) <= BF16 * np.abs(k) + 1e-5 * ka)
    assert np.all(np.abs(down(e["v"]) - v) <= BF16 * np.abs(v) + 1e-5 * va)


def test_offsets_past_32_bits_in_the_cache(dev):
    """A pool of more than 2^31 elements: rows appended to and expanded from its last pages."""
    import torch
    rng = np.random.default_rng(24)
    row, pages, n = 576, 60000, 100
    assert (pages - 3) * 64 * row > 2 ** 31
    cache = torch.empty(pages, 64, row, dtype=torch.bfloat16, device=dev)
    cache[-3:] = 0
    rows, table = bits(rng, n, row), np.array([[pages - 1, pages - 3]])
    slots = np.concatenate([(pages - 1) * 64 + np.arange(64), (pages - 3) * 64 + np.arange(n - 64)])
    p = K.make_params(1, 4, 1, 512, 64, 2, pages, 0)
    K.append_slots_tensor(K.KVATTN_MLA, p, up(rows, dev), None, i32(slots, dev), cache, 0.0)
    np.testing.assert_array_equal(down(cache[-1]), f64(rows[:64]))
    np.testing.assert_array_equal(down(cache[-3, :n - 64]), f64(rows[64:]))
    uk, uv = bits(rng, 4, 128, 512, scale=512 ** -0.5), bits(rng, 4, 512, 128, scale=512 ** -0.5)
    e = K.expand_kv_tensors(K.KVATTN_MLA, p, cache, i32(table, dev), i32([0, n], dev), up(uk, dev), up(uv, dev), n)
    k, v, ka, va = prompt.expand(f64(rows), f64(uk), f64(uv), 1)
    assert np.all(np.abs(down(e["k"]) - k) <= BF16 * np.abs(k) + 1e-5 * ka)
    assert np.all(np.abs(down(e["v"]) - v) <= BF16 * np.abs(v) + 1e-5 * va)


def test_offsets_past_32_bits_in_the_rows(dev):
    """Queries, keys, values and outputs of more than 2^31 elements; the sequence stands at their end."""
    import torch
    rng = np.random.default_rng(25)
    T, nq, nk = 8_500_000, 140, 300
    assert (T - nk) * 256 > 2 ** 31
    x = prefill_case(rng, 2, 2, 128, 0, 128, [nq], [nk], slack=0)

    def far(t, axis, shape):
        big = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        big.narrow(axis, T - t.shape[axis], t.shape[axis]).copy_(t)
        return big
    q = far(up(x["q"], dev), 0, (T, 2, 128))
    k, v = far(up(x["k"], dev), 1, (2, T, 128)), far(up(x["v"], dev), 1, (2, T, 128))
    got = K.prefill_tensors(q, None, k, None, v, i32([T - nq, T], dev), i32([T - nk, T], dev), 0.1)
    check_prefill(dict(out=got["out"][T - nq:], lse=got["lse"][T - nq:]), x, [nq], [nk], 0.1, True)


# ------------------------------------------------------------- all together

@pytest.mark.parametrize("name", ["mla", "gla", "mlra_128k"])
def test_a_prompt_then_tokens(dev, name):
    """Tables, append, expand and prefill of two chunks, then the last token of
    every sequence through the absorbed decode on the same cache: the expanded
    and the absorbed form of the same attention.  Both round keys or queries,
    weights, outputs to bf16 (each <= 2^-8 relative), four roundings apart:
    relative 2-norm within 1.5e-2, and both within 1e-2 of the fp64 chain."""
    import torch
    rng = np.random.default_rng(20)
    s = W.WORKLOADS[name]
    H, G, dc, dr, dh = 16, s.num_kv, s.d_nope, s.d_rope, 128
    B, mpps, pages = 3, 12, 40
    chunks = [[300, 1, 129], [64, 200, 0]]
    row = G * dc + dr
    variant = s.variant_id
    R = G if s.variant == "mlra" else 1            # branches: the output is the sum over them
    cache = torch.full((pages, 64, row), float("nan"), dtype=torch.bfloat16, device=dev)
    uk, uv = bits(rng, H, dh, R * dc, scale=dc ** -0.5), bits(rng, H, R * dc, dh, scale=dh ** -0.5)
    tuk, tuv = up(uk, dev), up(uv, dev)
    lens, table, count = i32([0] * B, dev), i32(np.full((B, mpps), -1), dev), i32([pages], dev)
    pool = i32(rng.permutation(pages), dev)
    scale = (dh + dr) ** -0.5
    past = [np.zeros((0, row))] * B
    err = word(dev)
    for new in chunks:
        T = sum(new)
        rows, q, qr = bits(rng, T, row), bits(rng, T, H, dh), bits(rng, T, H * R, dr)
        tq, tqr = up(q, dev), up(qr, dev)
        st = K.build_tables_tensors(lens, i32(new, dev), pool, count, table, T + 10, err, inplace=True)
        p = K.make_params(B, H, G, dc, dr, mpps, pages, 0)
        K.append_slots_tensor(variant, p, up(rows, dev), st["pos"][:T].contiguous(), st["slots"][:T].contiguous(), cache,
                              W.ROPE_BASE, err)
        K.rope_tensor(tqr, st["pos"], 0, dr, W.ROPE_BASE, H * R)
        total = int(st["kv_start"][-1])
        e = K.expand_kv_tensors(variant, p, cache, table, st["kv_start"], tuk, tuv, total, err)
        got = K.prefill_tensors(tq, tqr, e["k"], e["k_rope"], e["v"], st["q_start"], st["kv_start"], scale, device_error=err)
        total_out = got["out"].view(T, H, R, dh).double().sum(2)
        # the fp64 chain
        at, off, num, den = 0, 0.0, 0.0, 0.0
        from oracle import steps
        for b, n in enumerate(new):
            pos = len(past[b]) + np.arange(n)
            r = f64(rows[at:at + n])
            if n:
                r[:, G * dc:] = steps.rope(r[:, G * dc:], pos, W.ROPE_BASE)
            past[b] = np.concatenate([past[b], r])
            ref = np.zeros((H, n, dh))
            for r in range(R):
                cols = slice(r * dc, (r + 1) * dc) if R > 1 else slice(0, G * dc)
                wc = cols if R > 1 else slice(None)
                k, v, _, _ = prompt.expand(past[b][:, cols], f64(uk)[:, :, wc], f64(uv)[:, wc], 1 if R > 1 else G)
                for h in range(H if n else 0):
                    qq = np.concatenate([f64(q[at:at + n, h]), steps.rope(f64(qr[at:at + n, h * R + r]), pos, W.ROPE_BASE)], 1)
                    ref[h] += prompt.attention(qq, np.concatenate([k[h], past[b][:, G * dc:]], 1), v[h], scale, True)[0]
            num += ((down(total_out[at:at + n]).transpose(1, 0, 2) - ref) ** 2).sum()
            den += (ref ** 2).sum()
            at += n
        assert np.sqrt(num / den) <= 1e-2
    assert int(err.item()) == 0
    # the newest token of each sequence again, absorbed
    last = [0, chunks[1][0] + chunks[1][1] - 1]
    idx = torch.tensor([chunks[1][0] - 1, chunks[1][0] + chunks[1][1] - 1], device=dev)
    p = K.make_params(2, H, G, dc, dr, mpps, pages, 500, branch_out=1 if R > 1 else 0)
    qa = K.head_proj_tensor(tq[idx].contiguous(), tuk)
    ol = torch.empty(2, H, R * dc, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(2, H * R, dtype=torch.float32, device=dev)
    ws = torch.zeros(K.kvattn_workspace_size(variant, p), dtype=torch.uint8, device=dev)
    K.decode_tensors(variant, p, qa, tqr[idx].contiguous(), cache, table, lens, scale, ol, lse, ws)
    one = down(K.head_proj_tensor(ol, tuv))
    two = down(total_out[idx])
    assert len(last) == 2 and np.linalg.norm(one - two) <= 1.5e-2 * np.linalg.norm(two)
    # lse of the two forms: keys rounded to bf16 in one, the absorbed query in the other
    assert np.abs(down(lse) - down(got["lse"][idx])).max() <= 2e-2


# ------------------------------------------------- sizes of a first call

FRESH = """
import sys
import numpy as np, torch
from oracle import prompt
from shared_kv_caches_b200 import kvattn as K
B = int(sys.argv[1])
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda:0")
pages = B + 5
free = np.random.default_rng(B).permutation(pages)
table = np.full((B, 1), -1)
r = K.build_tables_tensors(i32([0] * B), i32([1] * B), i32(free), i32([pages]), i32(table), B)
ref = prompt.build_tables([0] * B, [1] * B, free, pages, table, B, pages)
ref.pop("err")
for k in ref:
    assert np.array_equal(r[k].cpu().numpy(), ref[k]), k
"""


@pytest.mark.parametrize("batch", [4072, 4073, 4095, 4096])
def test_tables_first_call_of_a_process(dev, batch):
    """Batches around the 48 KB of shared memory that a launch may take without an opt-in."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH, str(batch)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_of_several_host_threads(dev):
    """Expansions of two widths and tables of two batches at once, each thread with its own stream and buffers."""
    import threading

    import torch
    rng = np.random.default_rng(27)
    jobs = []
    for dc, batch in ((512, 9000), (64, 5000)):
        cache, table, uk, uv, p, mpps = expand_case(rng, dev, 2, 1, dc, 16, 64, 64, [100, 70])
        x = [up(cache, dev), i32(table, dev), i32(starts([100, 70]), dev), up(uk, dev), up(uv, dev)]
        one = i32([1] * batch, dev)
        pool = i32(np.arange(batch), dev)
        jobs.append((p, x, one, one * 0, pool, i32([batch], dev), i32(np.full((batch, 1), -1), dev), batch))
    torch.cuda.synchronize()
    want = [K.expand_kv_tensors(K.KVATTN_MLA, j[0], *j[1], 170)["k"].clone() for j in jobs]
    torch.cuda.synchronize()
    faults = []

    def work(j, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    got = K.expand_kv_tensors(K.KVATTN_MLA, j[0], *j[1], 170)
                    t = K.build_tables_tensors(j[3], j[2], j[4], j[5], j[6], j[7])
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got["k"], ref) and int(t["free_left"]) == 0
        except Exception as e:          # a thread's failure is the test's
            faults.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults, faults


# ------------------------------------- what the tables say of refused requests

@pytest.mark.parametrize("new,tokens,pages,want", [
    ([64] * 5, 64, 3, prompt.ERR_TOKENS),                       # one page taken, two left: only the tokens ran out
    ([64, 640], 64, 3, prompt.ERR_TOKENS | prompt.ERR_POOL),    # ten pages wanted of two
    ([64, 64, 64], 128, 1, prompt.ERR_TOKENS | prompt.ERR_POOL),
    ([64, 128, 0, 64], 64, 3, prompt.ERR_TOKENS),
    ([1] * 3000, 70, 2980, prompt.ERR_TOKENS),
])
def test_tables_refused_for_tokens_do_not_use_up_the_pool(dev, new, tokens, pages, want):
    rng = np.random.default_rng(28)
    cached, free = np.zeros(len(new), int), rng.permutation(pages)
    table = np.full((len(new), 10), -7)
    ref = prompt.build_tables(cached, new, free, pages, table, tokens, pages)
    assert ref["err"] == want
    same_tables(run_tables(dev, cached, new, table, free, pages, tokens), ref)


def test_tables_error_words_of_random_requests(dev):
    """Tokens, pages and table rows that run out at different requests."""
    rng = np.random.default_rng(29)
    seen = set()
    for _ in range(60):
        n = int(rng.integers(1, 40))
        cached, new = rng.integers(0, 150, n), rng.integers(0, 200, n) * (rng.random(n) < 0.8)
        table, free, count, pages = table_case(rng, cached, new, shrink=int(rng.integers(0, 40)) * int(rng.random() < 0.6))
        if rng.random() < 0.3:
            table = table[:, :max(table.shape[1] - 1, 1)]
            cached = np.minimum(cached, 64 * table.shape[1])
        m = max(int(new.sum()) + 5 - int(rng.integers(0, 600)) * int(rng.random() < 0.6), 0)
        ref = prompt.build_tables(cached, new, free, count, table, m, pages)
        seen.add(ref["err"])
        same_tables(run_tables(dev, cached, new, table, free, count, m), ref)
    assert {0, prompt.ERR_TOKENS, prompt.ERR_POOL, prompt.ERR_TOKENS | prompt.ERR_POOL} <= seen


@pytest.mark.parametrize("new", [9, 10, 11])
def test_tables_lengths_end_at_31_bits(dev, new):
    """A table with room for 2^31 tokens: a length of 2^31 - 1 is served, the next one is refused."""
    import torch
    table = torch.zeros(1, 1 << 25, dtype=torch.int32, device=dev)
    err = word(dev)
    r = K.build_tables_tensors(i32([2 ** 31 - 10], dev), i32([new], dev), i32(np.arange(9), dev), i32([0], dev), table, 16,
                               device_error=err)
    fits = new == 9
    assert int(err.item()) == (0 if fits else K.KVATTN_DEVERR_SEQ_TOO_LONG)
    assert int(r["seq_lens"]) == 2 ** 31 - 10 + (9 if fits else 0) and int(r["kv_start"][1]) == int(r["seq_lens"])
    want = [(2 ** 31 - 10 + i) % 64 for i in range(9)] if fits else [-1] * new
    assert r["slots"].tolist()[:len(want)] == want and r["slots"].tolist()[new:] == [-1] * (16 - new)


# ------------------------------------------------------ one turn for all calls

@pytest.mark.parametrize("top", [1 << 15, 1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("variant,kv,dn,dr", [("mla", 1, 64, 64), ("gqa", 2, 128, 0)])
def test_append_turns_exactly_as_rope_does(dev, top, variant, kv, dn, dr):
    """Bit for bit, near and far: the rounding of a far angle reaches the stored bits where the two form it apart."""
    import torch
    rng = np.random.default_rng(30)
    n = 30000
    pages, base = -(-n // 64), W.ROPE_BASE
    pos = i32(rng.integers(-(top // 8), top, n), dev)
    slots = i32(rng.permutation(pages * 64)[:n], dev)
    p = K.make_params(1, 2 * kv, kv, dn, dr, pages, pages, 0)
    if dr:
        rows = up(bits(rng, n, dn + dr), dev)
        cache = torch.zeros(pages, 64, dn + dr, dtype=torch.bfloat16, device=dev)
        K.append_slots_tensor(K.VARIANTS[variant], p, rows, pos, slots, cache, base)
        got = cache.view(-1, dn + dr)[slots.long()]
        K.rope_tensor(rows, pos, dn, dr, base, 1)
    else:
        rows = up(bits(rng, n, 2, kv * dn), dev)
        cache = torch.zeros(pages, 2, 64, kv * dn, dtype=torch.bfloat16, device=dev)
        K.append_slots_tensor(K.VARIANTS[variant], p, rows, pos, slots, cache, base)
        got = cache.transpose(1, 2).reshape(-1, 2, kv * dn)[slots.long()]
        keys = rows[:, 0].contiguous().view(n * kv, dn)
        K.rope_tensor(keys, pos, 0, dn, base, kv)
        rows[:, 0] = keys.view(n, kv * dn)
    assert torch.equal(got.view(torch.int16), rows.view(torch.int16))


def test_both_appends_store_the_same_bits(dev):
    import torch
    rng = np.random.default_rng(31)
    B, Q, row, mpps = 40, 64, 576, 600
    pages = B * Q
    rows = up(bits(rng, B, Q, row), dev)
    pos = np.array([rng.choice(mpps * 64, Q, replace=False) for _ in range(B)])
    table = np.zeros((B, mpps), int)
    for b in range(B):              # a page of its own for every page that a position falls in
        table[b, pos[b] // 64] = b * Q + np.arange(Q)
    slots = np.take_along_axis(table, pos // 64, 1) * 64 + pos % 64
    p = K.make_params(B, 8, 1, 512, 64, mpps, pages, mpps * 64, q_len=Q)
    one, two = (torch.zeros(pages, 64, row, dtype=torch.bfloat16, device=dev) for _ in range(2))
    t, ps, tab = i32(slots.reshape(-1), dev), i32(pos, dev), i32(table, dev)
    assert K.kvattn_append_kv(K.KVATTN_MLA, p, rows.data_ptr(), ps.data_ptr(), tab.data_ptr(), one.data_ptr(), W.ROPE_BASE, None,
                              torch.cuda.current_stream().cuda_stream) == 0
    K.append_slots_tensor(K.KVATTN_MLA, p, rows.view(-1, row), ps.view(-1), t, two, W.ROPE_BASE)
    assert torch.equal(one.view(torch.int16), two.view(torch.int16))


@pytest.mark.parametrize("reach", [1.0, 1e14, 1e18])
def test_prefill_scale_zero_weighs_every_key_the_same(dev, reach):
    """Whatever the scores are: below 2^127, so that the exponents stay below 2^-21.  A weight is 1 within 2^-21 and
    rounds to 1 in bf16; 270 fp32 additions are off by 270 * 2^-24 < 2^-15 of sum |v|, those of the denominator by as
    much: 2^-13 of the mean of |v| covers both, and the output's own rounding is 2^-8.  lse: 2^-15 of the denominator,
    2^-21 of the maximum and the logarithm's own 2^-22."""
    rng = np.random.default_rng(32)
    ql, kl = [140], [270]
    x = prefill_case(rng, 2, 2, 64, 0, 64, ql, kl)
    x["q"][:140] = W.f32_to_bf16_bits((f64(x["q"][:140]) * reach).astype(np.float32))
    x["k"][:, :270] = W.f32_to_bf16_bits((f64(x["k"][:, :270]) * reach).astype(np.float32))
    got = call(dev, x, ql, kl, 0.0, True)
    out, lse = down(got["out"])[:140], down(got["lse"])[:140]
    for h in range(2):
        v = f64(x["v"][h, :270])
        for i in range(140):
            n = i + 131
            want, mass = v[:n].mean(0), np.abs(v[:n]).mean(0)
            assert np.all(np.abs(out[i, h] - want) <= BF16 * np.abs(want) + 2.0 ** -13 * mass)
            assert abs(lse[i, h] - np.log(n)) <= 2.0 ** -14


# --------------------------------------------------- larger grids, first calls

@pytest.mark.parametrize("tokens", [4097, 20000, 40000])
def test_tables_in_place_with_many_tokens(dev, tokens):
    """Lengths and free count updated in place while other CTAs read them (a cluster from 4097 tokens on, and more
    tokens than its eight CTAs take at once): eager, then replayed in a graph."""
    import torch
    rng = np.random.default_rng(tokens)
    B = 37
    cached = rng.integers(0, 300, B)
    new = rng.multinomial(tokens - 3, np.full(B, 1 / B))
    steps = 4
    table, free, count, pages = table_case(rng, cached, steps * new, mpps=int(-(-(cached + steps * new).max() // 64)) + 1)
    lens, cnt, tab, one, pool = i32(cached, dev), i32([count], dev), i32(table, dev), i32(new, dev), i32(free, dev)
    err = word(dev)
    ref_c, ref_t, ref_n = cached, table, count

    def same(r):
        nonlocal ref_c, ref_t, ref_n
        torch.cuda.synchronize()
        ref = prompt.build_tables(ref_c, new, free, ref_n, ref_t, tokens, pages)
        assert ref.pop("err") == 0 == int(err.item())
        same_tables({k: v.cpu().numpy() for k, v in r.items()}, ref)
        ref_c, ref_t, ref_n = ref["seq_lens"], ref["block_table"], int(ref["free_left"][0])

    same(K.build_tables_tensors(lens, one, pool, cnt, tab, tokens, err, inplace=True))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = K.build_tables_tensors(lens, one, pool, cnt, tab, tokens, err, inplace=True)
    for _ in range(steps - 1):
        g.replay()
        same(r)


@pytest.mark.parametrize("H,G,dc,variant", [(20, 2, 64, "gla"), (14, 2, 128, "gla"), (5, 3, 64, "mlra"), (9, 1, 64, "mla")])
def test_expand_more_tile_pairs_than_clusters(dev, H, G, dc, variant):
    """Clusters that take whole tile pairs through every group and head pair, then runs of what is left."""
    import torch
    rng = np.random.default_rng(H)
    lens = [9000, 1, 0, 7000, 130, 129] + [64] * 40
    R = G if variant == "mlra" else 1
    cache, table, _, _, p, mpps = expand_case(rng, dev, H, G, dc, 16, 16, 24, lens)
    uk, uv = bits(rng, H, 16, R * dc, scale=dc ** -0.5), bits(rng, H, R * dc, 24, scale=dc ** -0.5)
    err = word(dev)
    x = (K.VARIANTS[variant], p, up(cache, dev), i32(table, dev), i32(starts(lens), dev), up(uk, dev), up(uv, dev), sum(lens), err)
    got = K.expand_kv_tensors(*x)
    assert int(err.item()) == 0
    again = K.expand_kv_tensors(*x)
    assert all(torch.equal(got[k].view(torch.int16), again[k].view(torch.int16)) for k in got)
    if R == 1:
        check_expand(got, cache, table, uk, uv, G, lens, mpps)
        return
    for r in range(R):
        cols = np.r_[r * dc:(r + 1) * dc, R * dc:R * dc + 16]
        one = dict(k=got["k"][r::R], v=got["v"][r::R], k_rope=got["k_rope"])
        check_expand(one, cache[..., cols], table, uk[..., r * dc:(r + 1) * dc], uv[:, r * dc:(r + 1) * dc], 1, lens, mpps)


CAPTURED = """
import numpy as np, torch
from shared_kv_caches_b200 import kvattn as K
dev = "cuda:0"
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
gen = torch.Generator(dev).manual_seed(0)
draw = lambda *s: torch.randn(*s, generator=gen, device=dev).to(torch.bfloat16)
T, H, pages = {tokens}, 4, {tokens} // 64 + 2
lens, new, pool, cnt, tab = i32([0, 0]), i32([T - 70, 70]), i32(np.arange(pages)), i32([pages]), i32(np.zeros((2, pages)))
rows, q, qr, uk, uv = draw(T, 80), draw(T, H, 64), draw(T, H, 16), draw(H, 64, 64), draw(H, 64, 64)
cache, err = torch.zeros(pages, 64, 80, dtype=torch.bfloat16, device=dev), i32([0])
p = K.make_params(2, H, 1, 64, 16, pages, pages, 0)

def step():
    t = K.build_tables_tensors(lens, new, pool, cnt, tab, T, err)
    K.append_slots_tensor(K.KVATTN_MLA, p, rows, t["pos"], t["slots"], cache, 1e4, err)
    e = K.expand_kv_tensors(K.KVATTN_MLA, p, cache, tab, t["kv_start"], uk, uv, T, err)
    return K.prefill_tensors(q, qr, e["k"], e["k_rope"], e["v"], t["q_start"], t["kv_start"], 0.1, device_error=err)

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
want = step()
assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]) and int(err) == 0
assert bool(torch.isfinite(got["out"]).all()) and float(got["out"].float().abs().max()) > 0
"""


@pytest.mark.parametrize("tokens", [300, 9000])
def test_a_process_whose_first_calls_are_captured(dev, tokens):
    """A whole step captured before any call ran eagerly, with and without the plan's launch."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURED.format(tokens=tokens)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_expand_and_append_at_once_on_two_streams(dev):
    """Expansions of the same cache on two streams with their own workspaces, beside appends to other pages."""
    import torch
    rng = np.random.default_rng(33)
    lens = [3000, 200]
    cache, table, uk, uv, p, mpps = expand_case(rng, dev, 4, 1, 128, 32, 64, 64, lens)
    free = np.setdiff1d(np.arange(cache.shape[0]), table)[0]
    x = (K.KVATTN_MLA, p, up(cache, dev), i32(table, dev), i32(starts(lens), dev), up(uk, dev), up(uv, dev), sum(lens))
    rows, pos, slots = up(bits(rng, 64, 160), dev), i32(np.arange(64), dev), i32(free * 64 + np.arange(64), dev)
    one = K.expand_kv_tensors(*x)
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            with torch.cuda.stream(s):
                got.append(K.expand_kv_tensors(*x))
        K.append_slots_tensor(K.KVATTN_MLA, p, rows, pos, slots, x[2], W.ROPE_BASE)
    torch.cuda.synchronize()
    for y in got:
        assert all(torch.equal(one[k].view(torch.int16), y[k].view(torch.int16)) for k in one)


def test_append_of_as_many_tokens_as_there_are_numbers(dev):
    """2^31 - 1 rows of 16 bytes, all but the last few skipped: the walk over them ends where they do."""
    import torch
    n = 2 ** 31 - 1
    rows = torch.empty(n, 8, dtype=torch.bfloat16, device=dev)
    slots = torch.full((n,), -1, dtype=torch.int32, device=dev)
    tail = torch.arange(24, device=dev).view(3, 8).to(torch.bfloat16)
    rows[-3:], slots[-3:] = tail, i32([5, 70, 127], dev)
    cache, err = torch.zeros(2, 64, 8, dtype=torch.bfloat16, device=dev), word(dev)
    p = K.make_params(1, 4, 1, 8, 0, 2, 2, 0)
    K.append_slots_tensor(K.KVATTN_MLA, p, rows, None, slots, cache, 0.0, err)
    want = torch.zeros(128, 8, dtype=torch.bfloat16, device=dev)
    want[[5, 70, 127]] = tail
    assert torch.equal(cache.view(128, 8), want) and int(err.item()) == 0


def test_prefill_axes_of_one_element_may_have_a_stride_of_zero(dev):
    """One head or one token, with the stride that a broadcast view gives its axis."""
    rng = np.random.default_rng(34)
    for ql, kl in (([1], [1]), ([5], [70])):
        x = prefill_case(rng, 1, 1, 64, 16, 64, ql, kl, slack=0)
        t = {k: up(v, dev) for k, v in x.items()}
        one = {k: v.as_strided(v.shape, [0 if n == 1 else s for n, s in zip(v.shape, v.stride())]) for k, v in t.items()}
        assert all(0 in v.stride() for k, v in one.items() if k != "kr")
        got = K.prefill_tensors(one["q"], one["qr"], one["k"], one["kr"], one["v"], i32(starts(ql), dev), i32(starts(kl), dev), 0.1)
        check_prefill(got, x, ql, kl, 0.1, True)


@pytest.mark.parametrize("low", [-1e37, 1e36, -3e9, 1.5 * 2.0 ** 29])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_rows_whose_scores_are_all_far_from_zero(dev, low, causal):
    """Every key that some rows attend scores the same number far from zero (a mask of a type's lowest value, written
    into the keys): those rows weigh their keys alike.  Scores are one exact product, the weights 1 up to 2^64 on both
    sides; 400 fp32 additions and the output's rounding as in the test of scale 0, the lse that of one rounding of the
    score (2^-22 of it).  Rows of the other head, with common scores, keep their bits."""
    rng = np.random.default_rng(35)
    nq, nk = 200, 400
    x = prefill_case(rng, 2, 2, 64, 0, 64, [nq], [nk])
    plain = call(dev, x, [nq], [nk], 0.125, causal)
    q, k = f64(x["q"]), f64(x["k"])
    q[:nq, 0], k[0, :nk] = 0.0, 0.0
    q[:nq, 0, 3], k[0, :nk, 3] = 2.0 ** 20, low / 2.0 ** 20 * 8
    x["q"], x["k"] = W.f32_to_bf16_bits(q.astype(np.float32)), W.f32_to_bf16_bits(k.astype(np.float32))
    score = 0.125 * f64(x["q"])[0, 0, 3] * f64(x["k"])[0, 0, 3]
    got = call(dev, x, [nq], [nk], 0.125, causal)
    out, lse, v = down(got["out"]), down(got["lse"]), f64(x["v"][0, :nk])
    for i in range(nq):
        n = i + nk - nq + 1 if causal else nk
        want, mass = v[:n].mean(0), np.abs(v[:n]).mean(0)
        assert np.all(np.abs(out[i, 0] - want) <= BF16 * np.abs(want) + 2.0 ** -13 * mass)
        assert abs(lse[i, 0] - (score + np.log(n))) <= 2.0 ** -22 * abs(score) + 2.0 ** -14
    assert np.array_equal(out[:nq, 1], down(plain["out"])[:nq, 1]) and np.array_equal(lse[:nq, 1], down(plain["lse"])[:nq, 1])
