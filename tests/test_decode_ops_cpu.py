"""attn_kv_append, attn_decode_step and token_sample without a GPU: what they
refuse, before any launch, and the 64-bit definitions that the GPU tests use."""
import ctypes

import numpy as np
import pytest

import _decode_ref as ref  # noqa: E402

M = 1 << 20


@pytest.fixture(scope="module")
def q():
    import quantized_expert_matvec_b200 as q
    return q


def cache(q, **kw):
    from quantized_expert_matvec_b200._binding import KVCacheDesc
    d = dict(k=M, v=2 * M, k_page_stride=2 * 16 * 128, v_page_stride=2 * 16 * 128, n_pages=8, page_size=16, n_kv=2,
             head_dim=128, dtype=q.QE_BF16, reserved=0)
    d.update(kw)
    return KVCacheDesc(*[d[n] for n, _ in KVCacheDesc._fields_])


def append(q, c=None, rope=None, T=2, n_q=4, qp=16 * M, kp=17 * M, vp=18 * M, dt=1, qs=512, ks=256, vs=256, out=19 * M,
           os=512, pos=None, kv_pos=20 * M, seq=None, table=21 * M, n_seq=2, stride=4, ws=22 * M, ws_bytes=4096):
    c = c if c is not None else cache(q)
    return q.lib.attn_kv_append(ctypes.byref(c), rope, T, n_q, qp, kp, vp, dt, qs, ks, vs, out, os, pos, kv_pos, seq,
                                table, n_seq, stride, ws, ws_bytes, None)


def attend(q, c=None, B=2, n_q=4, qp=16 * M, qs=512, prefix=None, prefix_len=0, table=21 * M, stride=4, kv_len=20 * M,
           out=19 * M, os=512, lse=None, ws=22 * M, ws_bytes=1 << 40, scale=0.1):
    c = c if c is not None else cache(q)
    return q.lib.attn_decode_step(ctypes.byref(c), B, n_q, qp, qs, prefix, prefix_len, table, stride, kv_len, scale, out,
                                  os, lse, ws, ws_bytes, None)


def sample(q, logits=M, dt=0, B=2, V=100, stride=100, t=None, k=None, p=None, m=None, u=2 * M, token=3 * M, lp=None):
    return q.lib.token_sample(logits, dt, B, V, stride, t, k, p, m, u, token, lp, None)


@pytest.mark.parametrize("kw,what", [
    (dict(dtype=0), "dtype"), (dict(head_dim=96), "head_dim"), (dict(page_size=0), "page_size"),
    (dict(page_size=65537), "page_size"), (dict(n_kv=0), "n_kv"), (dict(n_pages=-1), "n_pages"),
    (dict(k_page_stride=4095), "page strides"), (dict(v_page_stride=4100), "page strides"),
    (dict(k=None), "cache k is NULL"), (dict(v=2 * M + 8), "cache v is not 16-byte"),
])
def test_bad_caches_are_refused(q, kw, what):
    for call in (append, attend):
        assert call(q, cache(q, **kw)) == q.QE_ERR_INVALID_ARG
        assert what in q.qe_last_error()
    if not ("k" in kw or "v" in kw):
        assert q.lib.attn_workspace_bytes(ctypes.byref(cache(q, **kw)), 4, 2) == 0


@pytest.mark.parametrize("kw,what", [
    (dict(T=-1), "T must"), (dict(n_q=-1), "n_q"), (dict(dt=3), "in_dtype"), (dict(kp=None), "k is NULL"),
    (dict(vp=18 * M + 8), "v is not 16-byte"), (dict(qp=None), "q is NULL"), (dict(out=None), "q_out is NULL"),
    (dict(kv_pos=None), "kv_pos"), (dict(table=None), "table"), (dict(n_seq=-1), "n_seq"), (dict(qs=516), "strides"),
    (dict(ks=128), "strides"), (dict(os=256), "strides"), (dict(ws=None), "workspace"), (dict(ws=22 * M + 16), "workspace"),
    (dict(ws_bytes=255), "workspace"), (dict(out=16 * M + 16), "overlaps"), (dict(out=17 * M), "overlaps"),
    (dict(out=16 * M, dt=0), "overlaps"),  # in place needs one dtype
])
def test_append_refuses(q, kw, what):
    assert append(q, **kw) == q.QE_ERR_INVALID_ARG
    assert what in q.qe_last_error()


@pytest.mark.parametrize("kw,what", [
    (dict(rotary_dim=24), "rotary_dim"), (dict(rotary_dim=144), "rotary_dim"), (dict(n_axes=0), "n_axes"),
    (dict(n_axes=5), "n_axes"), (dict(inv_freq=None), "inv_freq"), (dict(n_axes=2), "pair_axis"),
])
def test_append_refuses_rotations(q, kw, what):
    from quantized_expert_matvec_b200._binding import RopeDesc
    axes = (ctypes.c_uint8 * 64)(*([0] * 63 + [2]))
    d = dict(inv_freq=M, pair_axis=ctypes.cast(axes, ctypes.POINTER(ctypes.c_uint8)), rotary_dim=128, n_axes=3,
             adjacent=0, reserved=0)
    d.update(kw)
    r = RopeDesc(*[d[n] for n, _ in RopeDesc._fields_])
    assert append(q, rope=ctypes.byref(r)) == q.QE_ERR_INVALID_ARG
    assert what in q.qe_last_error()


@pytest.mark.parametrize("kw", [
    dict(out=16 * M, kp=16 * M, ks=512),                                         # in place: k is q's first heads
    dict(out=16 * M, vp=16 * M + 512, vs=512),                                   # v its last ones
    dict(out=16 * M, kp=16 * M + 1024, ks=512),                                  # the next token's
    dict(out=16 * M, qs=1024, os=1024, kp=16 * M + 1792, ks=1024),               # k runs into the next token's q
    dict(out=16 * M, qs=1024, os=1024, vp=16 * M + 1024, vs=1032),               # another stride: they meet somewhere
    dict(out=16 * M + 1024, qs=1024, os=1024, kp=16 * M + 1536, ks=1024),        # k in a q_out beside q
    dict(T=1, out=16 * M, kp=16 * M + 768, ks=512),
])
def test_append_refuses_inputs_that_it_would_overwrite(q, kw):
    assert append(q, **kw) == q.QE_ERR_INVALID_ARG
    assert "overlaps" in q.qe_last_error()


@pytest.mark.parametrize("kw", [dict(qs=1024, os=1024, out=16 * M + 1008), dict(qs=1024, os=1024, out=16 * M + 1040),
                                dict(qs=1024, os=1032, out=16 * M + 1024), dict(qs=1024, os=1024, out=16 * M - 1008)])
def test_attention_refuses_outputs_on_queries(q, kw):
    assert attend(q, **kw) == q.QE_ERR_INVALID_ARG
    assert "overlaps" in q.qe_last_error()


@pytest.mark.parametrize("kw,what", [
    (dict(n_q=3), "n_q"), (dict(n_q=0), "n_q"), (dict(B=-1), "B must"), (dict(B=4097), "B must"),
    (dict(prefix_len=-1), "prefix_len"), (dict(prefix_len=1 << 30), "prefix_len"), (dict(prefix_len=5), "prefix_pages"),
    (dict(stride=-1), "table_stride"), (dict(stride=1 << 27), "table_stride"), (dict(table=None), "table"),
    (dict(kv_len=None), "kv_len"), (dict(qp=16 * M + 2), "q is not"), (dict(out=None), "out is NULL"),
    (dict(qs=520 + 4), "strides"), (dict(os=504), "strides"), (dict(out=16 * M + 512), "overlaps"),
    (dict(ws=None), "workspace"), (dict(ws=22 * M + 128), "workspace"), (dict(ws_bytes=1024), "too small"),
    (dict(lse=2), "lse"), (dict(scale=-0.1), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(scale=2.5e38), "scale"),  # its product with log2 e is infinite
])
def test_attention_refuses(q, kw, what):
    assert attend(q, **kw) == q.QE_ERR_INVALID_ARG
    assert what in q.qe_last_error()


@pytest.mark.parametrize("kw,what", [
    (dict(dt=7), "dtype"), (dict(B=-1), "B must"), (dict(V=0), "V must"), (dict(V=524289, stride=524289), "V must"),
    (dict(stride=99), "stride"), (dict(logits=None), "logits"), (dict(logits=M + 2), "logits"), (dict(u=None), "u is NULL"),
    (dict(token=None), "token"), (dict(t=M + 1), "temperature"), (dict(k=M + 1), "top_k"), (dict(p=M + 1), "top_p"),
    (dict(m=M + 1), "min_p"), (dict(lp=M + 1), "logprob"),
])
def test_sampling_refuses(q, kw, what):
    assert sample(q, **kw) == q.QE_ERR_INVALID_ARG
    assert what in q.qe_last_error()


def test_empty_calls_do_nothing(q):
    assert append(q, T=0, kp=None, vp=None, qp=None, out=None, kv_pos=None, table=None, ws=None) == q.QE_OK
    assert attend(q, B=0, qp=None, out=None, kv_len=None, table=None, ws=None) == q.QE_OK
    assert sample(q, B=0, logits=None, u=None, token=None) == q.QE_OK


def test_workspace_grows_with_the_batch_only(q):
    c = cache(q)
    sizes = [q.lib.attn_workspace_bytes(ctypes.byref(c), 4, b) for b in (1, 2, 64, 4096)]
    assert sizes[0] > 256 and sizes == sorted(sizes)


def test_binding_checks_before_the_library(q):
    import torch
    t = torch.zeros((2, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        q.KVCache(t, t)
    with pytest.raises(ValueError, match="n_pages, n_kv"):
        q.KVCache(t[0], t[0])
    with pytest.raises(ValueError, match="inv_freq"):
        q.Rope(torch.zeros(8))


def test_binding_names_what_is_missing(q):
    # the arguments with a default of None that a call cannot do without
    import torch
    t = torch.zeros((2, 2, 64))
    with pytest.raises(ValueError, match="ws is missing"):
        q.attn_kv_append(None, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="q_out is missing"):
        q.attn_kv_append(None, t, t, t, t, t, ws=t)
    with pytest.raises(ValueError, match="ws is missing"):
        q.attn_decode_step(None, t, t, t, t)


def test_reference_rotation_is_a_rotation():
    # lengths of the pairs stay, a quarter turn swaps them, no pair beyond rotary_dim moves
    rng = np.random.RandomState(0)
    x = rng.randn(3, 2, 32)
    f = np.array([np.pi / 2] + [0.3] * 7, np.float64)
    for adjacent in (False, True):
        y, _ = ref.rotate(x, np.array([[0, 1, 2]]), f, [0] * 8, adjacent)
        a, b = (0, 1) if adjacent else (0, 8)
        assert np.allclose(y[0], x[0]) and np.array_equal(y[:, :, 16:], x[:, :, 16:])
        assert np.allclose(y[1, :, a], -x[1, :, b]) and np.allclose(y[1, :, b], x[1, :, a])
        assert np.allclose(y[2, :, a], -x[2, :, a])
        assert np.allclose((y ** 2).sum(), (x ** 2).sum())


def test_reference_attention_special_cases():
    rng = np.random.RandomState(1)
    k, v = rng.randn(5, 8), rng.randn(5, 8)
    out, lse, _, _ = ref.attend(np.zeros((1, 8)), k, v, 1.0, "bf16")
    assert np.allclose(out[0], v.mean(axis=0)) and np.allclose(lse, np.log(5))
    out, _, _, _ = ref.attend(1e3 * k[2:3], k, v, 1.0, "bf16")
    assert np.allclose(out[0], v[np.argmax(k @ k[2])])


def test_reference_sampling_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [ref.sample(x, u)[0] for u in (0.0, 0.05, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [ref.sample(x, u, top_k=2)[0] for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]
    assert [ref.sample(x, u, top_p=0.65)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert [ref.sample(x, u, min_p=0.6)[0] for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert ref.sample(x, 0.7, temperature=0.0) == (1, 0.0)
    assert abs(ref.sample(x, 0.0, top_k=2)[1] - np.log(4 / 7)) < 1e-12
