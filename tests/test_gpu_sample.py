"""token_sample on the GPU against its 64-bit definition: tokens equal, log
probabilities within the rounding of the result; and a decode step of the
operators together."""
import math

import numpy as np
import pytest

import _decode_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q(cuda):
    import quantized_expert_matvec_b200 as q
    return q


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def run(q, logits, u, **kw):
    import torch
    B = logits.shape[0]
    token = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 7.0, device="cuda")
    kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32)
    args = {n: torch.tensor(kw[n], dtype=t, device="cuda") for n, t in kinds.items() if kw.get(n) is not None}
    q.token_sample(logits, torch.as_tensor(u, dtype=torch.float32).cuda(), token, logprob=lp, **args)
    return token.cpu().numpy(), lp.cpu().numpy()


def check(logits, u, token, lp, **kw):
    x = logits.double().cpu().numpy()
    V = x.shape[1]
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    for b in range(len(x)):
        row = {n: kw[n][b] if n == "top_k" else f32(kw[n][b]) for n in ("temperature", "top_k", "top_p", "min_p")
               if kw.get(n) is not None}
        want, want_lp = ref.sample(x[b], f32(u[b]), **row)
        assert token[b] == want, (b, row, f32(u[b]), token[b], want)
        # ln(w / Z) of weights rounded to 2^-S of the largest (S >= 43 for V <= 2^19), then to fp32
        if want >= 0 and want_lp > -20:
            assert abs(lp[b] - want_lp) <= 2.0 ** -24 * abs(want_lp) + (V + math.exp(20)) * 2.0 ** -43, (b, lp[b], want_lp)
        elif want < 0:
            assert lp[b] == -math.inf


def rows(B, V, dtype, seed, spread=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = spread * torch.randn((B, V), generator=g, device="cuda")
    n = min(V, 20)
    x.scatter_add_(1, torch.randint(0, V, (B, n), generator=g, device="cuda"),
                   6.0 * torch.rand((B, n), generator=g, device="cuda"))
    return x.to(dt(dtype))


SHAPES = [(1, 1, "f32"), (3, 2, "bf16"), (5, 7, "f16"), (9, 1000, "f32"), (4, 8193, "bf16"), (3, 32000, "f16"),
          (2, 100003, "bf16"), (2, 131072, "f32"), (2, 262145, "f32"), (1, 524288, "f32"), (1, 524287, "f16")]


@pytest.mark.parametrize("B,V,dtype", SHAPES, ids=[f"{b}x{v}_{d}" for b, v, d in SHAPES])
def test_each_filter_and_all_together(q, cuda, B, V, dtype):
    x = rows(B, V, dtype, 1)
    rng = np.random.RandomState(2)
    k = [max(1, int(V ** rng.rand())) for _ in range(B)]
    for kw in (dict(), dict(top_k=k), dict(top_p=list(0.3 + 0.69 * rng.rand(B))), dict(min_p=list(0.2 * rng.rand(B))),
               dict(temperature=list(0.2 + 2 * rng.rand(B)), top_k=k, top_p=list(0.5 + 0.5 * rng.rand(B)),
                    min_p=list(0.1 * rng.rand(B)))):
        for trial in range(3):
            u = rng.rand(B).astype(np.float32)
            token, lp = run(q, x, u, **kw)
            check(x, u, token, lp, **kw)


def test_unaligned_rows(q, cuda):
    # rows that start at every element offset, an odd distance apart
    import torch
    for dtype in ("f32", "bf16"):
        B, V = 6, 1003
        flat = rows(1, 8 + B * 1009, dtype, 3)[0]
        for off in range(9 if dtype == "bf16" else 5):
            x = torch.as_strided(flat, (B, V), (1009, 1), off)
            kw = dict(top_k=[1, 2, 30, 500, 1002, 1003], top_p=[0.9] * 6)
            u = np.linspace(0, 0.999, B).astype(np.float32)
            token, lp = run(q, x, u, **kw)
            check(x, u, token, lp, **kw)


def test_ties_go_to_the_lower_index(q, cuda):
    import torch
    # all equal: top-k and top-p keep the lowest indices, exactly
    for V, dtype in ((1000, "bf16"), (65536, "f32"), (100003, "f16")):
        x = torch.zeros((6, V), device="cuda").to(dt(dtype))
        u = np.array([0.0, 0.25, 0.5, 0.75, 0.999, 0.9999999], np.float32)
        for kw in (dict(), dict(top_k=[7] * 6), dict(top_p=[0.5] * 6), dict(min_p=[1.0] * 6), dict(top_k=[100] * 6, top_p=[0.25] * 6)):
            token, lp = run(q, x, u, **kw)
            check(x, u, token, lp, **kw)
    # a few values only, so that every cut falls into a tie; -0 and +0 are one value
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-2, 3, (8, 5003), generator=g, device="cuda").float()
    x = torch.where((x == 0) & (torch.rand(x.shape, generator=g, device="cuda") < 0.5), -0.0, x)
    kw = dict(top_k=[1, 10, 900, 1100, 2000, 3000, 5002, 5003], top_p=[1.0, 0.5, 0.9, 0.3, 0.99, 0.7, 0.6, 0.2])
    for s in range(4):
        u = np.random.RandomState(s).rand(8).astype(np.float32)
        token, lp = run(q, x, u, **kw)
        check(x, u, token, lp, **kw)


def test_masked_infinite_and_nan_logits(q, cuda):
    import torch
    V = 9001
    x = rows(8, V, "f32", 5)
    ban = torch.rand((8, V), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") < 0.97
    x[0] = torch.where(ban[0], -math.inf, x[0])
    x[1] = torch.where(ban[1], torch.finfo(torch.float32).min, x[1])
    x[2] = -math.inf
    x[3] = math.nan
    x[4] = torch.where(ban[4], math.nan, x[4])
    x[5, [17, 4000, 8000]] = math.inf
    x[6] = torch.finfo(torch.float32).min
    x[7, 5000] = torch.finfo(torch.float32).max
    for kw in (dict(), dict(top_k=[500] * 8, top_p=[0.8] * 8), dict(top_p=[0.6] * 8, min_p=[0.3] * 8),
               dict(temperature=[0.0] * 8), dict(top_k=[8990] * 8)):
        for s in range(3):
            u = np.random.RandomState(s).rand(8).astype(np.float32)
            token, lp = run(q, x, u, **kw)
            check(x, u, token, lp, **kw)
            assert token[2] == -1 and token[3] == -1


def test_edges_of_the_settings(q, cuda):
    x = rows(1, 5000, "f32", 7).expand(10, -1).contiguous()
    nan = math.nan
    kw = dict(temperature=[1.0, -1.0, nan, 1e-30, 1e30, math.inf, 1.0, 1.0, 0.7, 1e-44],
              top_k=[0, 5, 5, 0, 0, 0, -3, 5000, 6000, 0],
              top_p=[0.0, 0.5, 0.5, 1.0, 1.0, 1.0, -1.0, 1.5, 1e-40, 0.9],
              min_p=[0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 2.0, -1.0, 0.0])
    for u in (0.0, 0.3, 0.99999994, 1.0, 2.0, -1.0):
        us = np.full(10, u, np.float32)
        token, lp = run(q, x, us, **kw)
        check(x, us, token, lp, **kw)
    token, _ = run(q, x, np.full(10, nan, np.float32), top_p=[nan] * 10, min_p=[nan] * 10)
    want, _ = run(q, x, np.zeros(10, np.float32))
    assert np.array_equal(token, want)


def test_close_logits_around_zero_and_wide_ranges(q, cuda):
    # logits whose difference to the largest is the same fp32 number although they differ;
    # ranges of hundreds, and of a millionth
    import torch
    g = torch.Generator(device="cuda").manual_seed(8)
    V = 20000
    x = torch.empty((5, V), device="cuda")
    x[0] = torch.randn(V, generator=g, device="cuda") * 1e-9
    x[0, 77] = 4.0
    x[1] = torch.randn(V, generator=g, device="cuda") * 300
    x[2] = 1.0 + torch.rand(V, generator=g, device="cuda") * 1e-6
    x[3] = -100.0 - torch.rand(V, generator=g, device="cuda")
    x[4] = torch.randn(V, generator=g, device="cuda") * 1e-40
    kw = dict(top_k=[9000, 50, 333, 19999, 4000], top_p=[0.99, 0.9, 0.5, 0.75, 0.6])
    for s in range(4):
        u = np.random.RandomState(s).rand(5).astype(np.float32)
        for kk in (kw, dict(top_k=kw["top_k"]), dict(top_p=kw["top_p"])):
            token, lp = run(q, x, u, **kk)
            check(x, u, token, lp, **kk)


def test_a_row_does_not_depend_on_its_batch(q, cuda):
    x = rows(40, 30011, "bf16", 9)
    u = np.random.RandomState(1).rand(40).astype(np.float32)
    kw = dict(top_k=[40] * 40, top_p=[0.9] * 40, temperature=[0.7] * 40)
    token, lp = run(q, x, u, **kw)
    check(x, u, token, lp, **kw)
    for b in (0, 17, 39):
        t, l = run(q, x[b:b + 1].clone(), u[b:b + 1], **{n: v[:1] for n, v in kw.items()})
        assert t[0] == token[b] and l[0] == lp[b]


@pytest.mark.parametrize("dtype,V,pad", [("f32", 90001, 3), ("bf16", 200003, 0), ("f16", 170000, 5)])
def test_many_large_rows(q, cuda, dtype, V, pad):
    # so many rows that they are read in passes instead of kept on chip: all settings side by
    # side, masked, equal, infinite and NaN logits among them, rows that start off any boundary
    import torch
    B = 150
    flat = torch.zeros(B * (V + pad) + 1, device="cuda", dtype=dt(dtype))
    x = torch.as_strided(flat, (B, V), (V + pad, 1), 1 if pad else 0)
    x.copy_(rows(B, V, dtype, 12))
    ban = torch.rand((B, V), generator=torch.Generator(device="cuda").manual_seed(13), device="cuda") < 0.5
    x[3::10] = torch.where(ban[3::10], -math.inf, x[3::10])
    x[4::10] = torch.where(ban[4::10], math.nan, x[4::10])
    x[5::30] = 1.5                      # all equal
    x[15::30] = x[15::30].round()       # a few values
    x[25::30, 77:V:1000] = math.inf
    x[9] = -math.inf
    rng = np.random.RandomState(3)
    b = np.arange(B)
    kw = dict(temperature=np.where(b % 7 == 3, 0.0, 0.3 + 1.5 * rng.rand(B)),
              top_k=np.where(b % 3 == 0, np.exp(rng.uniform(0, np.log(V), B)).astype(int), 0),
              top_p=np.where(b % 2 == 0, 0.3 + 0.7 * rng.rand(B), 1.0), min_p=np.where(b % 5 == 1, 0.1 * rng.rand(B), 0.0))
    kw = {n: list(v) for n, v in kw.items()}
    kw["top_k"] = [int(k) for k in kw["top_k"]]
    for s in range(2):
        u = np.random.RandomState(20 + s).rand(B).astype(np.float32)
        token, lp = run(q, x, u, **kw)
        check(x, u, token, lp, **kw)
    # the same rows a few at a time (kept on chip) choose the same tokens
    few = slice(60, 66)
    t, l = run(q, x[few].clone(), u[few], **{n: v[few] for n, v in kw.items()})
    assert np.array_equal(t, token[few]) and np.array_equal(l, lp[few])


def test_streamed_rows_of_the_largest_vocabulary(q, cuda):
    # so many rows of 524288 logits that they are read in passes, most logits of a row in one
    # bin of the histogram: sums over more logits than 32 bits hold for 16-bit pieces of the weights
    import torch
    B, V = 40, 524288
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.empty((B, V), device="cuda")
    kw = dict(temperature=[1.0] * B, top_p=[0.0] * B)
    for b in range(B):
        x[b] = -0.01 - 0.037 * b                                     # one value: bins 0 .. a few hundred
        kw["top_p"][b] = 0.3 + 0.69 * (b * 0.618 % 1)
        if b % 4 == 1:
            x[b] += 0.05 * torch.rand(V, generator=g, device="cuda")  # near one another
        elif b % 4 == 2:
            x[b] = -40.0 - 10 * torch.rand(V, generator=g, device="cuda")  # the last bin
            kw["temperature"][b] = 60.0
        x[b, (1009 * b + 7) % V] = 0.1
    x[3] = torch.where(torch.rand(V, generator=g, device="cuda") < 0.4, -math.inf, x[3])
    for keep in (None, [int(V * (0.2 + 0.019 * b)) for b in range(B)]):
        kk = dict(kw, top_k=keep) if keep else kw
        u = np.random.RandomState(22).rand(B).astype(np.float32)
        token, lp = run(q, x, u, **kk)
        check(x, u, token, lp, **kk)
        few = slice(18, 20)  # kept on chip: the same tokens
        t, l = run(q, x[few].clone(), u[few], **{n: v[few] for n, v in kk.items()})
        assert np.array_equal(t, token[few]) and np.array_equal(l, lp[few])


@pytest.mark.parametrize("V", [2, 900, 2048, 2049, 5000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_differences_beyond_the_type(q, cuda, V, dtype):
    # a token forced by the type's largest value over masks of its lowest: their difference is infinite
    import torch
    top, low = torch.finfo(dt(dtype)).max, torch.finfo(dt(dtype)).min
    x = torch.full((8, V), low, device="cuda").to(dt(dtype))
    for b in range(8):
        x[b, (b * 37 + 1) % V] = top
    x[5:, V // 2:] = -math.inf
    x[6, 0] = 3.0
    for kw in (dict(), dict(top_k=[1, 2, 3, 50, V - 1, 7, 2, 2]), dict(top_k=[2] * 8, top_p=[0.9] * 8), dict(top_p=[0.5] * 8),
               dict(min_p=[0.1] * 8), dict(top_k=[3] * 8, min_p=[0.5] * 8),
               dict(temperature=[math.inf, 1e38, 2e38, 3e38, 1e37, 1e38, math.inf, 1e38]),
               dict(temperature=[math.inf, 1e38, 2e38, 3e38, 1e37, 1e38, math.inf, 1e38], top_k=[2] * 8)):
        for s in range(3):
            u = np.random.RandomState(s).rand(8).astype(np.float32)
            token, lp = run(q, x, u, **kw)
            check(x, u, token, lp, **kw)


def test_outputs_beside_the_batch_stay(q, cuda):
    import torch
    x = rows(4, 777, "f32", 10)
    token = torch.full((6,), -9, dtype=torch.int32, device="cuda")
    q.token_sample(x, torch.rand(4, device="cuda"), token[1:5])
    assert token[0] == -9 and token[5] == -9 and bool((token[1:5] >= 0).all())


def test_binding_refuses(q, cuda):
    import torch
    x, u, t = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="dense rows"):
        q.token_sample(x.t().contiguous().t(), u, t)
    with pytest.raises(ValueError, match="float32, bfloat16"):
        q.token_sample(x.double(), u, t)
    with pytest.raises(ValueError, match="token"):
        q.token_sample(x, u, t.long())
    with pytest.raises(ValueError, match="top_p"):
        q.token_sample(x, u, t, top_p=torch.zeros(3, device="cuda"))
    with pytest.raises(q.QEError, match="stride"):
        q.token_sample(torch.zeros(8, device="cuda").expand(2, 8), u, t)


def test_a_decode_step_of_all_operators(q, cuda):
    """Three tokens through rotation + append, attention behind a shared prefix,
    the MoE layer step and the choice of a token: eagerly and as one captured
    graph, bit for bit; the attention also against its definition."""
    import torch
    from _util import dev_router, fill_pool
    B, n_q, n_kv, D, page, prefix, V, H, E, K, I = 4, 4, 2, 64, 16, 40, 1000, 256, 16, 2, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    cfg = q.Cfg(H, E, K, I, 64, 1e-6)
    pool = q.ExpertPool(cfg, E, 4)
    fill_pool(pool, 0, 0)
    W = dev_router(0, 0, E, H)
    layer = q.Layer(W.data_ptr(), None, None, pool.table.data_ptr())
    ws = q.workspace(cfg, B)
    qkv = torch.randn((3, B, (n_q + 2 * n_kv) * D), generator=g, device="cuda")
    head = (torch.randn((H, V), generator=g, device="cuda") / 16)
    us = torch.rand((3, B), generator=g, device="cuda")
    inv = torch.rand(D // 2, generator=g, device="cuda")
    kp0 = torch.randn((20, n_kv, page, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(4, 4 + 2 * B, dtype=torch.int32, device="cuda").reshape(B, 2)
    pp = torch.arange(3, dtype=torch.int32, device="cuda")

    def fresh():
        s = dict(kp=kp0.clone(), vp=-kp0, kv_pos=torch.tensor([14, 0, 15, 3], dtype=torch.int32, device="cuda"),
                 qo=torch.zeros((B, n_q, D), dtype=torch.bfloat16, device="cuda"),
                 o=torch.zeros((B, n_q, D), dtype=torch.bfloat16, device="cuda"),
                 y=torch.zeros((3, B, H), device="cuda"), x=torch.zeros((B, H), device="cuda"),
                 logits=torch.zeros((B, V), device="cuda"), token=torch.zeros((3, B), dtype=torch.int32, device="cuda"))
        s["kc"] = q.KVCache(s["kp"], s["vp"])
        s["ws"] = q.attn_workspace(s["kc"], n_q, B)
        s["rope"] = q.Rope(inv)
        s["pos"] = (s["kv_pos"] + prefix).reshape(1, B).contiguous()
        s["len"] = s["kv_pos"] + 1
        return s

    def token(s, t):
        x = qkv[t]
        q.attn_kv_append(s["kc"], x[:, :n_q * D].unflatten(1, (n_q, D)),
                         x[:, n_q * D:(n_q + n_kv) * D].unflatten(1, (n_kv, D)),
                         x[:, (n_q + n_kv) * D:].unflatten(1, (n_kv, D)), table, s["kv_pos"], s["qo"], rope=s["rope"],
                         pos=s["pos"], ws=s["ws"])
        q.attn_decode_step(s["kc"], s["qo"], s["o"], table, s["len"], pp, prefix, None, None, s["ws"])
        s["x"].copy_(s["o"].view(B, n_q * D))
        q.moe_layer_step(cfg, layer, s["x"], s["y"][t], True, ws=ws)
        torch.mm(s["y"][t] / (1 + s["y"][t].abs().amax()), head, out=s["logits"])
        q.token_sample(s["logits"], us[t], s["token"][t], top_k=s["topk"])
        s["kv_pos"] += 1
        s["pos"] += 1
        s["len"] += 1

    eager = fresh()
    eager["topk"] = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    for t in range(3):
        token(eager, t)
        if t == 2:
            kp, vp, qq = (eager[n].double().cpu().numpy() for n in ("kp", "vp", "qo"))
            o, ln, tb = eager["o"].double().cpu().numpy(), (eager["len"] - 1).tolist(), table.cpu().numpy()
            for b in range(B):
                for h in range(n_kv):
                    k, v = (np.concatenate([ref.gather(p, page, [0, 1, 2], prefix, h), ref.gather(p, page, tb[b], ln[b], h)])
                            for p in (kp, vp))
                    want, _, tol, _ = ref.attend(qq[b, 2 * h:2 * h + 2], k, v, D ** -0.5, "bf16")
                    assert np.all(np.abs(o[b, 2 * h:2 * h + 2] - want) <= tol)
    torch.cuda.synchronize()
    for b in range(B):
        want, _ = ref.sample(eager["logits"][b].double().cpu().numpy(), float(us[2, b]), top_k=50)
        assert int(eager["token"][2, b]) == want
    s = fresh()
    s["topk"] = eager["topk"]
    st = torch.cuda.Stream()
    start = [s[n].clone() for n in ("kv_pos", "pos", "len")]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for t in range(3):
            token(s, t)
    for _ in range(2):  # the second replay starts over and gives the same
        for n, v in zip(("kv_pos", "pos", "len"), start):
            s[n].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("kp", "vp", "o", "y", "token"):
            assert torch.equal(s[n], eager[n]), n
    assert q.qe_workspace_status(s["ws"]) == q.QE_OK and q.qe_workspace_status(ws) == q.QE_OK
