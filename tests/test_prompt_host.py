"""The prompt side without a GPU: what its entry points refuse before anything
is launched (the fake pointers are never dereferenced), their workspace sizes,
the helpers' checks, and the fp64 reference against brute force."""

import numpy as np
import pytest

from oracle import prompt, steps
from shared_kv_caches_b200 import build as B
from shared_kv_caches_b200 import kvattn as K

FAKE = 1 << 20
INVALID, UNSUPPORTED, SMALL, MISALIGNED = (K.KVATTN_ERR_INVALID_ARG, K.KVATTN_ERR_UNSUPPORTED,
                                           K.KVATTN_ERR_WORKSPACE_TOO_SMALL, K.KVATTN_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return K.load()


# ------------------------------------------------------------------ tables
TABLE_PTRS = ["cached", "new", "free", "count", "table", "lens", "left", "q_start", "kv_start", "pos", "slots"]


def tables(batch=4, mpps=8, pages=100, tokens=64, **kw):
    ptr = {n: FAKE for n in TABLE_PTRS + ["err"]} | kw
    return K.kvattn_build_tables(batch, mpps, pages, tokens, *[ptr[n] for n in TABLE_PTRS + ["err"]], None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(mpps=0), INVALID), (dict(pages=0), INVALID), (dict(tokens=-1), INVALID),
    (dict(batch=16385), UNSUPPORTED), (dict(pages=1 << 25), UNSUPPORTED), (dict(tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(pos=None), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 2), MISALIGNED), (dict(err=FAKE + 1), MISALIGNED),
])
def test_tables_refusals(lib, kw, status):
    assert tables(**kw) == status


@pytest.mark.parametrize("name", [n for n in TABLE_PTRS if n not in ("kv_start", "pos", "slots")])
def test_tables_null_pointers(lib, name):
    assert tables(**{name: None}) == INVALID


# ------------------------------------------------------------------ append
def append(variant=K.KVATTN_MLA, n=4, base=1e4, p=None, new=FAKE, pos=FAKE, slots=FAKE, cache=FAKE, err=None, **kw):
    d = dict(batch=1, num_q_heads=16, num_kv=1, d_nope=512, d_rope=64, max_pages_per_seq=4, num_pages=9, max_seq_len=0)
    d.update(kw)
    return K.kvattn_append_slots(variant, K.make_params(**d), new, n, pos, slots, cache, base, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(new=None), INVALID), (dict(slots=None), INVALID), (dict(cache=None), INVALID),
    (dict(pos=None), INVALID), (dict(base=0.5), INVALID), (dict(base=float("nan")), INVALID), (dict(base=float("inf")), INVALID),
    (dict(new=FAKE + 8), MISALIGNED), (dict(cache=FAKE + 8), MISALIGNED), (dict(slots=FAKE + 2), MISALIGNED),
    (dict(pos=FAKE + 2), MISALIGNED), (dict(err=FAKE + 2), MISALIGNED), (dict(num_pages=1 << 25), UNSUPPORTED),
    (dict(d_rope=60), UNSUPPORTED), (dict(num_kv=2), INVALID), (dict(cache_dtype=1), UNSUPPORTED),
    (dict(variant=K.KVATTN_GTA, d_nope=128, d_rope=0), INVALID),                    # tied rows are not turned
    (dict(variant=9), UNSUPPORTED), (dict(n=0), 0),
])
def test_append_refusals(lib, kw, status):
    assert append(**kw) == status


# ------------------------------------------------------------------ expand
EXPAND_PTRS = ["cache", "table", "start", "uk", "uv", "k", "v", "kr", "ws"]


def expand(variant=K.KVATTN_MLA, n=5000, d_k=128, d_v=128, ws_bytes=1 << 30, err=None, ptr=None, **kw):
    d = dict(batch=2, num_q_heads=16, num_kv=1, d_nope=512, d_rope=64, max_pages_per_seq=4, num_pages=9, max_seq_len=0)
    d.update(kw)
    x = {k: FAKE for k in EXPAND_PTRS} | (ptr or {})
    return K.kvattn_expand_kv(variant, K.make_params(**d), x["cache"], x["table"], x["start"], n, d_k, d_v, x["uk"], x["uv"],
                              x["k"], x["v"], x["kr"], x["ws"], ws_bytes, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(d_k=0), INVALID), (dict(d_k=132), UNSUPPORTED), (dict(d_k=136), UNSUPPORTED),
    (dict(d_v=60), UNSUPPORTED), (dict(d_nope=72), UNSUPPORTED), (dict(ws_bytes=100), SMALL),
    (dict(variant=K.KVATTN_GTA, d_rope=0), UNSUPPORTED), (dict(variant=K.KVATTN_GQA, d_rope=0), UNSUPPORTED),
    (dict(ptr=dict(ws=FAKE + 16)), MISALIGNED), (dict(err=FAKE + 2), MISALIGNED), (dict(n=0), 0),
    (dict(batch=16385), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED), (dict(n=2 ** 31 - 2), UNSUPPORTED),
])
def test_expand_refusals(lib, kw, status):
    assert expand(**kw) == status


@pytest.mark.parametrize("name", ["cache", "start", "uk", "uv", "k", "v", "kr", "ws"])
def test_expand_null_and_misaligned_pointers(lib, name):
    assert expand(ptr={name: None}) == INVALID
    assert expand(ptr={name: FAKE + 2}) == MISALIGNED


# ----------------------------------------------------------------- prefill
def params(**kw):
    d = dict(batch=2, num_q_heads=8, num_kv_heads=4, d_nope=128, d_rope=64, d_v=128, max_q_tokens=5000, max_kv_tokens=7000,
             causal=1, out_dtype=0, num_q_nope_heads=0)
    d.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    p = K.kvattn_prefill_params(*d.values())
    for k, v in kw.items():
        if k == "k_rope_stride":
            p.k_rope_stride = v
        elif k.endswith("stride"):
            setattr(p, k, (K.ctypes.c_int64 * 2)(*v))
    return p


PREFILL_PTRS = ["q", "qr", "k", "kr", "v", "qs", "ks", "out", "ws"]


def prefill(scale=0.1, lse=FAKE, err=None, ws_bytes=1 << 30, ptr=None, **kw):
    x = {k: FAKE for k in PREFILL_PTRS} | (ptr or {})
    return K.kvattn_prefill(params(**kw), x["q"], x["qr"], x["k"], x["kr"], x["v"], x["qs"], x["ks"], scale, x["out"], lse,
                            x["ws"], ws_bytes, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=3), INVALID), (dict(d_nope=0), INVALID),
    (dict(d_rope=-8), INVALID), (dict(d_v=0), INVALID), (dict(causal=2), INVALID), (dict(out_dtype=5), INVALID),
    (dict(num_q_nope_heads=3), INVALID), (dict(num_q_nope_heads=-1), INVALID), (dict(max_q_tokens=-1), INVALID), (dict(max_kv_tokens=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(d_nope=100), UNSUPPORTED), (dict(d_nope=256), UNSUPPORTED), (dict(d_rope=72), UNSUPPORTED), (dict(d_v=136), UNSUPPORTED),
    (dict(batch=16385), UNSUPPORTED), (dict(max_q_tokens=2 ** 31 - 1, num_q_heads=65535, num_kv_heads=1), UNSUPPORTED),
    (dict(ws_bytes=255), SMALL), (dict(lse=FAKE + 2), MISALIGNED), (dict(err=FAKE + 2), MISALIGNED),
    (dict(max_q_tokens=2 ** 31 - 2, num_q_heads=1, num_kv_heads=1), UNSUPPORTED), (dict(max_kv_tokens=2 ** 31 - 2), UNSUPPORTED),
    (dict(k_stride=(4, 128)), INVALID), (dict(v_stride=(-8, 128)), INVALID), (dict(out_stride=(1 << 38, 8)), INVALID),
    (dict(q_rope_stride=(12, 8)), INVALID), (dict(k_rope_stride=20), INVALID), (dict(max_q_tokens=0), 0),
])
def test_prefill_refusals(lib, kw, status):
    assert prefill(**kw) == status


@pytest.mark.parametrize("name", PREFILL_PTRS)
def test_prefill_null_and_misaligned_pointers(lib, name):
    assert prefill(ptr={name: None}) == INVALID
    assert prefill(ptr={name: FAKE + 2}) == MISALIGNED


def test_workspace_sizes_cover_a_tile_for_every_sequence(lib):
    assert K.kvattn_prefill_workspace_size(params(batch=3, max_q_tokens=5121)) >= 32 * (21 + 3)
    p = K.make_params(5, 16, 1, 512, 64, 4, 9, 0)
    assert K.kvattn_expand_workspace_size(K.KVATTN_MLA, p, 12900) >= 32 * (101 + 5)


def test_small_batches_need_no_workspace(lib):
    """Up to 32 sequences and 16 tiles (and, for attention, an item for each SM at most)."""
    p = K.make_params(5, 16, 1, 512, 64, 4, 9, 0)
    assert K.kvattn_expand_workspace_size(K.KVATTN_MLA, p, 128 * 11) == 0
    assert K.kvattn_expand_workspace_size(K.KVATTN_MLA, p, 128 * 11 + 1) > 0
    assert K.kvattn_prefill_workspace_size(params(max_q_tokens=256 * 14)) == 0
    assert K.kvattn_prefill_workspace_size(params(max_q_tokens=256 * 14 + 1)) > 0
    assert K.kvattn_prefill_workspace_size(params(max_q_tokens=256, num_q_heads=64)) > 0
    assert K.kvattn_prefill_workspace_size(params(batch=33, max_q_tokens=33, num_q_heads=4)) > 0


def test_workspace_sizes_refuse_what_the_calls_refuse(lib):
    p = K.make_params(5, 16, 1, 512, 64, 4, 9, 0)
    with pytest.raises(K.KvattnError):
        K.kvattn_expand_workspace_size(K.KVATTN_MLA, p, -1)


def test_helpers_check_shapes_and_types(lib):
    import torch
    z = torch.zeros
    bf = dict(dtype=torch.bfloat16)
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        K.prefill_tensors(z(4, 2, 64, **bf), None, z(2, 4, 64, **bf), None, z(2, 5, 64, **bf), z(2, **i), z(2, **i), 0.1)
    with pytest.raises(ValueError):
        K.prefill_tensors(z(4, 2, 64), None, z(2, 4, 64, **bf), None, z(2, 4, 64, **bf), z(2, **i), z(2, **i), 0.1)
    with pytest.raises(ValueError):
        K.build_tables_tensors(z(3, **i), z(2, **i), z(9, **i), z(1, **i), z(3, 4, **i), 5)
    p = K.make_params(1, 8, 1, 64, 16, 2, 2, 0)
    with pytest.raises(ValueError):
        K.append_slots_tensor(K.KVATTN_MLA, p, z(3, 72, **bf), z(3, **i), z(3, **i), z(2, 64, 80, **bf), 0.0)
    with pytest.raises(ValueError):
        K.append_slots_tensor(K.KVATTN_MLA, p, z(3, 80, **bf), z(3, **i), z(3, **i), z(2, 64, 72, **bf), 0.0)
    with pytest.raises(ValueError):
        K.expand_kv_tensors(K.KVATTN_MLA, p, z(2, 64, 80, **bf), z(1, 2, **i), z(2, **i), z(8, 32, 72, **bf), z(8, 64, 32, **bf), 9)


# --------------------------------------------------------- the reference
def test_reference_tables_place_every_token_once():
    rng = np.random.default_rng(0)
    cached, new = rng.integers(0, 200, 20), rng.integers(0, 200, 20)
    held = -(-cached // 64)
    perm = rng.permutation(200)
    table = np.full((20, 8), -1)
    at = 0
    for b in range(20):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.concatenate([perm[at:], np.full(at, -1)])
    r = prompt.build_tables(cached, new, free, 200 - at, table, int(new.sum()) + 3, 200)
    assert r["err"] == 0
    used = r["slots"][:new.sum()]
    assert len(set(used)) == len(used) and (r["slots"][new.sum():] == -1).all()
    for b in range(20):
        need = -(-(cached[b] + new[b]) // 64)
        mine = r["block_table"][b, :need]
        for i in range(new[b]):
            t = r["q_start"][b] + i
            assert r["pos"][t] == cached[b] + i and used[t] == mine[r["pos"][t] // 64] * 64 + r["pos"][t] % 64
    taken = [int(p) for b in range(20) for p in r["block_table"][b, held[b]:-(-(cached[b] + new[b]) // 64)]]
    assert taken == [int(p) for p in perm[at:][::-1][:len(taken)]] and r["free_left"][0] == 200 - at - len(taken)


def test_reference_attention_against_a_masked_matrix():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 8)), rng.standard_normal((9, 8)), rng.standard_normal((9, 4))
    s = 0.3 * q @ k.T
    s[np.arange(9)[None] > np.arange(5)[:, None] + 4] = -np.inf
    p = np.exp(s) / np.exp(s).sum(1, keepdims=True)
    out, lse, mass, reach = prompt.attention(q, k, v, 0.3, True)
    np.testing.assert_allclose(out, p @ v)
    np.testing.assert_allclose(lse, np.log(np.exp(s).sum(1)))
    np.testing.assert_allclose(mass, p @ np.abs(v))
    out, lse, _, _ = prompt.attention(q, k[:2], v[:2], 0.3, True)      # three queries without keys
    assert (out[:3] == 0).all() and np.isinf(lse[:3]).all() and np.isfinite(lse[3:]).all()
    np.testing.assert_allclose(out[3], v[0])


def test_reference_expansion_is_the_absorbed_score():
    """q . (W_UK c) = (q W_UK) . c, and P (c W_UV) = (P c) W_UV, group by group."""
    rng = np.random.default_rng(2)
    rows, uk, uv = rng.standard_normal((7, 2 * 6 + 4)), rng.standard_normal((4, 5, 6)), rng.standard_normal((4, 6, 3))
    k, v, _, _ = prompt.expand(rows, uk, uv, 2)
    q, w = rng.standard_normal((4, 5)), rng.random((7,))
    for h in range(4):
        c = rows[:, (h // 2) * 6:(h // 2) * 6 + 6]
        np.testing.assert_allclose(k[h] @ q[h], c @ (q[h] @ uk[h]))
        np.testing.assert_allclose(w @ v[h], (w @ c) @ uv[h])


def test_reference_append_turns_only_the_named_columns():
    rng = np.random.default_rng(3)
    cache, rows = rng.standard_normal((2, 64, 10)), rng.standard_normal((3, 10))
    out = prompt.append_rows(cache, rows, [7, 8, 9], [5, -1, 70], [(6, 4)], 100.0)
    np.testing.assert_array_equal(out[0, 5, :6], rows[0, :6])
    np.testing.assert_allclose(out[1, 6, 6:], steps.rope(rows[2, 6:], np.array(9), 100.0))
    keep = np.ones((2, 64), bool)
    keep[0, 5] = keep[1, 6] = False
    np.testing.assert_array_equal(out[keep], cache[keep])
