"""Host-side validation under random input (CPU only) of the norm + rotation,
shared-prefix and block entry points: any combination of sizes, types, strides
and pointers gives a documented status and never crashes.  Fake device
pointers, so this runs only where no GPU is present."""
import ctypes

import pytest
from hypothesis import given, settings, strategies as st

import kv_cache_attention_states_b200 as kca
from tests.test_abi_fuzz_cpu import CODES, CTX, DT, I32, I64, PTR, SCALE, WSB, _arr, vp


@pytest.fixture(scope="module", autouse=True)
def _no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake device pointers: CPU-only test")


AXES = st.one_of(st.none(), st.lists(st.integers(0, 255), min_size=128, max_size=128), st.just([i % 3 for i in range(128)]))
# mostly sound arguments, so that the later checks and the plans are reached
OK_PTR = st.one_of(st.just(0x10000), PTR)
OK_DT = st.one_of(st.sampled_from([kca.F32, kca.F16, kca.BF16]), DT)
GEOM = st.one_of(st.just((8, 1, 256)), st.tuples(I32, I32, I32))


@settings(max_examples=500, deadline=None, derandomize=True)
@given(q=OK_PTR, qs=st.one_of(st.just(2048), I64), k=OK_PTR, ks=st.one_of(st.just(256), I64), v=OK_PTR, ind=OK_DT,
       n=I32, flags=st.integers(-1, 4), wq=PTR, wk=PTR, wd=OK_DT, w0=SCALE, eps=SCALE, pos=OK_PTR, n_axes=I32, axis=AXES,
       inv=OK_PTR, qo=OK_PTR, qod=OK_DT, kc=OK_PTR, vc=OK_PTR, kd=OK_DT, rows=I64, dst=PTR, dst0=I64, ws=PTR)
def test_norm_rope_append(q, qs, k, ks, v, ind, n, flags, wq, wk, wd, w0, eps, pos, n_axes, axis, inv, qo, qod, kc, vc,
                          kd, rows, dst, dst0, ws):
    ax = None if axis is None else (ctypes.c_uint8 * 128)(*axis)
    assert kca.lib().attn_norm_rope_append(vp(q), qs, vp(k), ks, vp(v), ks, ind, n, flags, vp(wq), vp(wk), wd, w0, eps,
                                           vp(pos), n_axes, ax, vp(inv), vp(qo), qod, vp(kc), vp(vc), kd, rows, vp(dst),
                                           dst0, vp(ws), None) in CODES


@settings(max_examples=500, deadline=None, derandomize=True)
@given(q=OK_PTR, qd=OK_DT, pk=OK_PTR, pv=OK_PTR, prefix=I64, k=OK_PTR, v=OK_PTR, kd=OK_DT, geom=GEOM, cap=I64, ctx=CTX,
       batch=I32, dev=st.one_of(st.just(0), PTR), bound=I64, window=I32, scale=SCALE, out=OK_PTR, od=OK_DT, ws=OK_PTR,
       wsb=WSB, near=st.booleans(), host=st.booleans())
def test_decode_prefix(q, qd, pk, pv, prefix, k, v, kd, geom, cap, ctx, batch, dev, bound, window, scale, out, od, ws,
                       wsb, near, host):
    if near and 0 <= prefix <= 131072:
        ctx, cap, bound = [prefix + abs(c) % 100 for c in ctx], 100, prefix + 100
    arr, ptr = _arr(ctx)
    n = min(batch, len(arr)) if batch > 0 else batch
    lib = kca.lib()
    assert lib.attn_decode_prefix(vp(q), qd, vp(pk), vp(pv), prefix, vp(k), vp(v), kd, *geom, cap, n,
                                  ptr if host else None, vp(dev), bound, window, scale, vp(out), od, vp(ws), wsb,
                                  None) in CODES
    got = lib.attn_decode_prefix_workspace_bytes(qd, kd, prefix, n, ptr, window)
    assert got == 0 or got >= kca.WORKSPACE_HEADER


@settings(max_examples=500, deadline=None, derandomize=True)
@given(q=OK_PTR, qd=OK_DT, k=OK_PTR, v=OK_PTR, kd=OK_DT, geom=GEOM, cap=I64, batch=I32, codes=OK_PTR, scales=OK_PTR,
       bcap=I64, blocks=OK_PTR, n=I32, sink=I32, recent=I32, ctx=OK_PTR, bound=I64, n_new=I64, scale=SCALE, out=OK_PTR,
       od=OK_DT, ws=OK_PTR, wsb=WSB)
def test_blocks(q, qd, k, v, kd, geom, cap, batch, codes, scales, bcap, blocks, n, sink, recent, ctx, bound, n_new,
                scale, out, od, ws, wsb):
    lib = kca.lib()
    assert lib.attn_summarize_blocks(vp(k), kd, cap, batch, vp(ctx), n_new, vp(codes), vp(scales), vp(ws), None) in CODES
    assert lib.attn_select_blocks(vp(q), qd, vp(codes), vp(scales), bcap, batch, vp(ctx), bound, n, sink, recent,
                                  vp(blocks), vp(ws), wsb, None) in CODES
    assert lib.attn_decode_blocks(vp(q), qd, vp(k), vp(v), kd, *geom, cap, batch, vp(blocks), n, vp(ctx), bound, scale,
                                  vp(out), od, vp(ws), wsb, None) in CODES
    for got in (lib.attn_select_blocks_workspace_bytes(batch, bound), lib.attn_decode_blocks_workspace_bytes(batch, n)):
        assert got == 0 or got >= kca.WORKSPACE_HEADER
