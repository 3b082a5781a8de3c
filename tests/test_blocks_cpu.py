"""Host checks of the block calls that need no GPU, and pins of their oracle:
refusals come back before any CUDA call; the score bounds every key's product;
the oracle's attention over all blocks is plain attention."""
import numpy as np
import pytest

import kv_cache_attention_states_b200 as kca
import oracle
from oracle import blocks as ob

P = 1 << 20   # never dereferenced: every call here is refused on the host
NULL, GEOM, DTYPE, RANGE, WS, ALIGN = -1, -2, -3, -4, -5, -6


def _with(defaults, kw):
    assert not set(kw) - set(defaults)
    return list({**defaults, **kw}.values())


def _summarize(**kw):
    return kca.lib().attn_summarize_blocks(*_with(dict(k=P, kv=kca.F16, cap=640, batch=2, ctx=P, n_new=1, codes=P,
                                                       scales=P, ws=None, stream=None), kw))


def _select(**kw):
    return kca.lib().attn_select_blocks(*_with(dict(
        q=P, qd=kca.F32, codes=P, scales=P, cap=10, batch=2, ctx=P, bound=640, n=4, sink=1, recent=1, blocks=P, ws=P,
        ws_bytes=1 << 30, stream=None), kw))


def _decode(**kw):
    return kca.lib().attn_decode_blocks(*_with(dict(
        q=P, qd=kca.F16, k=P, v=P, kv=kca.F16, hq=8, hkv=1, d=256, cap=640, batch=2, blocks=P, n_list=4, ctx=P,
        bound=640, scale=0.0625, out=P, od=kca.F32, ws=P, ws_bytes=1 << 30, stream=None), kw))


@pytest.mark.parametrize("kw,code", [
    ({"k": None}, NULL), ({"ctx": None}, NULL), ({"codes": None}, NULL), ({"scales": None}, NULL),
    ({"kv": kca.I8}, DTYPE), ({"kv": -1}, DTYPE), ({"cap": 0}, RANGE), ({"cap": 131073}, RANGE), ({"batch": 0}, RANGE),
    ({"batch": 257}, RANGE), ({"n_new": 0}, RANGE), ({"n_new": 641}, RANGE),
    ({"k": P + 8}, ALIGN), ({"codes": P + 4}, ALIGN), ({"scales": P + 2}, ALIGN), ({"ctx": P + 4}, ALIGN),
    ({"ws": P + 2}, ALIGN)])
def test_summarize_refusals(kw, code):
    assert _summarize(**kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, NULL) for n in ("q", "codes", "scales", "ctx", "blocks", "ws")],
    ({"qd": 9}, DTYPE), ({"batch": 0}, RANGE), ({"batch": 257}, RANGE), ({"bound": 0}, RANGE), ({"bound": 131073}, RANGE),
    ({"cap": 8}, RANGE), ({"cap": 2049}, RANGE), ({"n": 0}, RANGE), ({"n": 2049}, RANGE), ({"sink": -1}, RANGE),
    ({"recent": 0}, RANGE), ({"sink": 4}, RANGE), ({"recent": 4}, RANGE), ({"sink": 2 ** 31 - 1}, RANGE),
    ({"recent": 2 ** 31 - 1}, RANGE), ({"q": P + 8}, ALIGN), ({"codes": P + 8}, ALIGN), ({"scales": P + 1}, ALIGN),
    ({"ctx": P + 4}, ALIGN), ({"blocks": P + 2}, ALIGN), ({"ws": P + 128}, WS), ({"ws_bytes": 24832}, WS)])
def test_select_refusals(kw, code):
    assert _select(**kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, NULL) for n in ("q", "k", "v", "ctx", "blocks", "out", "ws")],
    ({"hq": 4}, GEOM), ({"hkv": 2}, GEOM), ({"d": 128}, GEOM),
    ({"qd": 9}, DTYPE), ({"kv": kca.I8}, DTYPE), ({"od": kca.BF16}, DTYPE), ({"qd": kca.F32, "od": kca.F16}, DTYPE),
    ({"cap": 0}, RANGE), ({"cap": 131073}, RANGE), ({"batch": 0}, RANGE), ({"batch": 257}, RANGE), ({"bound": -1}, RANGE),
    ({"bound": 641}, RANGE), ({"n_list": 0}, RANGE), ({"n_list": 2049}, RANGE), ({"scale": 0.0}, RANGE),
    ({"scale": float("nan")}, RANGE), ({"scale": float("inf")}, RANGE), ({"scale": -1.0}, RANGE),
    ({"q": P + 8}, ALIGN), ({"k": P + 8}, ALIGN), ({"v": P + 8}, ALIGN), ({"out": P + 8}, ALIGN), ({"ctx": P + 4}, ALIGN),
    ({"blocks": P + 2}, ALIGN), ({"ws": P + 128}, WS)])
def test_decode_refusals(kw, code):
    assert _decode(**kw) == code


def test_workspace_queries_refuse_bad_sizes():
    L = kca.lib()
    for batch, bound in ((0, 5), (257, 5), (1, 0), (1, 131073)):
        assert L.attn_select_blocks_workspace_bytes(batch, bound) == 0
    assert L.attn_select_blocks_workspace_bytes(256, 131072) >= kca.WORKSPACE_HEADER + 256 * 2048 * 4
    for batch, n in ((0, 5), (257, 5), (1, 0), (1, 2049)):
        assert L.attn_decode_blocks_workspace_bytes(batch, n) == 0


def test_oracle_score_bounds_every_key_of_a_block():
    rng = np.random.default_rng(0)
    k = rng.standard_normal((1, 640, 256)).astype(np.float32)
    q = rng.standard_normal((8, 256)).astype(np.float32)
    codes, scales = ob.summarize(k, "f32", [640], 640, np.zeros((1, 10, 2, 256), np.int8), np.zeros((1, 10), np.float32))
    s = ob.scores(q, "f32", codes[0], scales[0], 10)
    exact = (q.astype(np.float64) @ k[0].T.astype(np.float64)).reshape(8, 10, 64).max((0, 2))
    # the codes are off by half a step each: at most (|q| sk + |k| sq + sq sk / 2) / 2 a dim
    sq = np.abs(q).max() / 127
    slack = 0.5 * (np.abs(q).sum(1).max() * scales[0].max() + 256 * np.abs(k).max() * sq + 256 * sq * scales[0].max())
    assert (s >= exact - slack).all()
    # exact bounds (no codes) dominate without slack
    hi, lo = k[0].reshape(10, 64, 256).max(1), k[0].reshape(10, 64, 256).min(1)
    u = (np.maximum(q, 0).astype(np.float64) @ hi.T + np.minimum(q, 0).astype(np.float64) @ lo.T).max(0)
    assert (u >= exact - 1e-9).all()


def test_oracle_attention_over_all_blocks_is_plain_attention():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 200, 256)).astype(np.float16)
    q = rng.standard_normal((8, 256)).astype(np.float32)
    for ctx in (1, 64, 150, 200):
        got, _, _ = ob.attend(q, "f32", k, v, "f16", [1, 3, 0, 2, -1], ctx)
        want = oracle.attention(q[None], k, v, np.array([ctx - 1]), q_dtype="f32", kv_dtype="f16")[0]
        assert np.abs(got - want).max() < 1e-12
    assert not ob.attend(q, "f32", k, v, "f16", [-1], 100)[0].any()


def test_oracle_choice_by_hand():
    codes = np.zeros((5, 2, 256), np.int8)
    codes[:, 0, 0] = [1, 5, 9, 5, 2]
    q = np.zeros((8, 256), np.float32)
    q[:, 0] = 127
    args = q, "f32", codes, np.ones(5, np.float32), 5 * 64
    assert ob.select(*args, 3) == [0, 2, 4]
    assert ob.select(*args, 4) == [0, 1, 2, 4]          # 1 before its equal, 3
    assert ob.select(*args, 3, 0, 1) == [1, 2, 4]
    assert ob.select(*args, 3, 0, 2) == [2, 3, 4]
    assert ob.select(*args, 7) == [0, 1, 2, 3, 4, -1, -1]
