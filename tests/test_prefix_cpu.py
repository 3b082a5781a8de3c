"""Host checks of attn_decode_prefix that need no GPU, and pins of its oracle."""
import ctypes

import numpy as np
import pytest

import kv_cache_attention_states_b200 as kca
import oracle
from oracle import prefix as op

P = 1 << 20   # never dereferenced: every call here is refused on the host
NULL, GEOM, DTYPE, RANGE, WS, ALIGN = -1, -2, -3, -4, -5, -6


def _ctx(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _call(**kw):
    a = dict(q=P, qd=kca.F16, pk=P, pv=P, prefix=100, k=P, v=P, kv=kca.F16, hq=8, hkv=1, d=256, cap=50, batch=2,
             ctx=_ctx(100, 150), dev=None, bound=0, window=0, scale=0.0625, out=P, od=kca.F32, ws=P, ws_bytes=1 << 40,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return kca.lib().attn_decode_prefix(*a.values())


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, NULL) for n in ("q", "pk", "pv", "k", "v", "ctx", "out", "ws")],
    ({"hq": 4}, GEOM), ({"hkv": 2}, GEOM), ({"d": 128}, GEOM),
    ({"qd": 9}, DTYPE), ({"kv": kca.I8}, DTYPE), ({"od": kca.BF16}, DTYPE), ({"qd": kca.F32, "od": kca.F16}, DTYPE),
    ({"dev": P, "bound": 150}, RANGE), ({"prefix": -1}, RANGE), ({"prefix": 131073}, RANGE), ({"cap": 0}, RANGE),
    ({"cap": 131073}, RANGE), ({"batch": 0}, RANGE), ({"batch": 257}, RANGE), ({"scale": 0.0}, RANGE),
    ({"scale": float("nan")}, RANGE), ({"scale": float("inf")}, RANGE),
    ({"ctx": _ctx(99, 150)}, RANGE), ({"ctx": _ctx(100, 151)}, RANGE), ({"ctx": _ctx(-1, 100)}, RANGE),
    ({"prefix": 131072, "ctx": _ctx(131072, 131073)}, RANGE),
    ({"ctx": None, "dev": P, "bound": 99}, RANGE), ({"ctx": None, "dev": P, "bound": 151}, RANGE),
    *[({n: P + 8}, ALIGN) for n in ("q", "pk", "pv", "k", "v", "out")],
    ({"ctx": None, "dev": P + 4, "bound": 150}, ALIGN), ({"ws": P + 128}, WS)])
def test_refusals(kw, code):
    assert _call(**kw) == code


def test_workspace_query_refuses_bad_sizes():
    f = kca.lib().attn_decode_prefix_workspace_bytes
    for qd, kd, prefix, batch, ctx in ((9, 1, 10, 1, _ctx(20)), (1, 3, 10, 1, _ctx(20)), (1, 1, -1, 1, _ctx(20)),
                                       (1, 1, 131073, 1, _ctx(131073)), (1, 1, 10, 0, _ctx(20)),
                                       (1, 1, 10, 257, _ctx(*[20] * 257)), (1, 1, 10, 1, None), (1, 1, 10, 1, _ctx(9)),
                                       (1, 1, 10, 1, _ctx(131073))):
        assert f(qd, kd, prefix, batch, ctx, 0) == 0


def test_oracle_is_plain_attention_over_the_joined_rows():
    rng = np.random.default_rng(3)
    pk, pv = rng.standard_normal((2, 90, 256)).astype(np.float16)
    k, v = rng.standard_normal((2, 40, 256)).astype(np.float16)
    q = rng.standard_normal((8, 256)).astype(np.float32)
    for ctx in (90, 91, 130):
        for window in (0, 1, 20, 60, 500):
            got = op.attend(q, "f32", pk, pv, k, v, "f16", ctx, window)[0]
            want = oracle.attention(q[None], np.concatenate((pk, k)), np.concatenate((pv, v)), np.array([ctx - 1]),
                                    window=window, q_dtype="f32", kv_dtype="f16")[0]
            assert np.abs(got - want).max() < 1e-12
    assert not op.attend(q, "f32", pk[:0], pv[:0], k, v, "f16", 0)[0].any()
