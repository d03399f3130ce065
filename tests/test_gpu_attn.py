"""attn_kv_append and attn_decode_step on the GPU against their 64-bit
definitions (_decode_ref), element by element within bounds that count the
roundings (derived there), and the calls' conventions: padding rows, bad pages,
strides, graphs, streams."""
import math

import numpy as np
import pytest

import _decode_ref as ref

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def q(cuda):
    import quantized_expert_matvec_b200 as q
    return q


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- append

APPEND = [
    # src, cache, T, n_q, n_kv, D, rd, axes, adjacent, page, far
    ("bf16", "bf16", 1, 4, 2, 128, 128, 1, False, 16, 100),
    ("f32", "bf16", 7, 6, 2, 64, 64, 1, True, 1, 5),
    ("f32", "f16", 33, 8, 1, 256, 64, 3, False, 24, 1000003),
    ("f16", "f16", 5, 3, 3, 128, 96, 2, True, 5, 2147480000),
    ("bf16", "f16", 130, 40, 8, 128, 16, 4, False, 64, 70000),
    ("f16", "bf16", 9, 1, 1, 64, 0, 1, False, 128, 9),
    ("f32", "f16", 3, 70, 7, 256, 256, 1, False, 65536, 131072),
]


def append_inputs(c, seed):
    import torch
    src, cache, T, n_q, n_kv, D, rd, axes, adjacent, page, far = c
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed)
    x = torch.randn((T, (n_q + 2 * n_kv) * D + 8), generator=g, device="cuda").to(dt(src))  # strided tokens
    n_seq = max(1, T // 3)
    cols = 2 if page > 1000 else (T + 3 * page) // page + 1
    places = rng.permutation(n_seq * cols * min(page, 64))[:T]  # distinct
    seq, kv_pos = places % n_seq, (places // n_seq)
    n_pages = n_seq * cols + 2
    d = dict(q=x[:, :n_q * D].unflatten(1, (n_q, D)), k=x[:, n_q * D:(n_q + n_kv) * D].unflatten(1, (n_kv, D)),
             v=x[:, (n_q + n_kv) * D:(n_q + 2 * n_kv) * D].unflatten(1, (n_kv, D)))
    if page > 1000:
        n_seq, n_pages = 1, 3
        seq, kv_pos = np.zeros(T, np.int64), page - 2 + np.arange(T)
        d["table"] = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    else:
        d["table"] = torch.from_numpy(rng.permutation(n_pages)[:n_seq * cols].reshape(n_seq, cols).astype(np.int32)).cuda()
    if T > 4:
        kv_pos[2] = -1
        kv_pos[T - 1] = -2147483648
    d["seq"] = torch.from_numpy(seq.astype(np.int32)).cuda()
    d["kv_pos"] = torch.from_numpy(kv_pos.astype(np.int32)).cuda()
    d["pos"] = torch.from_numpy(rng.randint(0, far + 1, (axes, T)).astype(np.int32)).cuda()
    for n in ("kp", "vp"):
        d[n] = torch.full((n_pages, n_kv, page, D), 3.0, device="cuda").to(dt(cache))
    d["out"] = torch.full((T, n_q, D), -5.0, device="cuda").to(dt(cache))
    half = rd // 2
    d["axis"] = [i % axes for i in range(half)]
    d["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).to(torch.float32).cuda()
    return d


def check_append(c, d):
    src, cache, T, n_q, n_kv, D, rd, axes, adjacent, page, far = c
    kv_pos, seq, table = (d[n].cpu().numpy() for n in ("kv_pos", "seq", "table"))
    pos, f = d["pos"].cpu().numpy(), d["inv_freq"].cpu().numpy()
    want_q, size_q = ref.rotate(host(d["q"]), pos, f, d["axis"], adjacent)
    want_k, size_k = ref.rotate(host(d["k"]), pos, f, d["axis"], adjacent)
    want_v = host(d["v"])

    def close(got, want, size):
        # sine and cosine are off by at most 2^-23 (the reduced angle's rounding and the
        # polynomial), two products and a sum by U32 each; then half a step of the cache's type
        e = (2.0 ** -23 + 2 * ref.U32) * size
        tol = e + ref.HALF_STEP[cache] * (np.abs(want) + e) + ref.TINY[cache]
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)

    live = kv_pos >= 0
    out = host(d["out"])
    close(out[live], want_q[live], size_q[live])
    assert np.all(out[~live] == -5.0)
    for got, want, size in ((host(d["kp"]), want_k, size_k), (host(d["vp"]), want_v, np.zeros_like(want_v))):
        touched = np.zeros((got.shape[0], page), bool)
        for t in np.nonzero(live)[0]:
            p = table[seq[t], kv_pos[t] // page]
            close(got[p, :, kv_pos[t] % page], want[t], size[t])
            touched[p, kv_pos[t] % page] = True
        assert np.all(got.transpose(0, 2, 1, 3)[~touched] == 3.0)


@pytest.mark.parametrize("c", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append_matches_the_definition(q, cuda, c):
    d = append_inputs(c, 3)
    kc = q.KVCache(d["kp"], d["vp"])
    ws = q.attn_workspace(kc, c[3], 1)
    rope = q.Rope(d["inv_freq"], d["axis"], c[8], n_axes=c[7]) if c[6] else q.Rope(d["inv_freq"], n_axes=c[7])
    q.attn_kv_append(kc, d["q"], d["k"], d["v"], d["table"], d["kv_pos"], d["out"], rope=rope, pos=d["pos"],
                     seq=d["seq"], ws=ws)
    assert q.qe_workspace_status(ws) == q.QE_OK
    check_append(c, d)


def exact_angle(pos, f):
    """pos * f reduced by the nearest multiple of 2 pi, from whole numbers (f is an fp32 number)."""
    from fractions import Fraction
    two_pi = Fraction(2 * 31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    a = Fraction(int(pos)) * Fraction(float(f))
    return float(a - round(a / two_pi) * two_pi)


def test_angles_of_far_positions(q, cuda):
    # positions and frequencies whose product has more bits than fp64: q is a unit vector, so that
    # q_out is cosine and sine themselves
    import torch
    rng = np.random.RandomState(23)
    T, D = 200, 64
    half = D // 2
    pos = np.concatenate([rng.randint(2 ** 30, 2 ** 31 - 1, T - 3), [2 ** 31 - 1, 2 ** 30 + 1, 1]]).astype(np.int32)
    f = np.concatenate([rng.uniform(0.5, 1.0, half // 2), np.exp(rng.uniform(0, math.log(16000), half // 2))]).astype(np.float32)
    x = torch.zeros((T, 1, D), device="cuda")
    x[:, :, :half] = 1.0
    kp = torch.zeros((T, 1, 8, D), dtype=torch.float16, device="cuda")
    kc = q.KVCache(kp, torch.zeros_like(kp))
    out = torch.zeros((T, 1, D), dtype=torch.float16, device="cuda")
    table = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    ws = q.attn_workspace(kc, 1, 1)
    q.attn_kv_append(kc, x, x, x, table, torch.zeros(T, dtype=torch.int32, device="cuda"), out,
                     rope=q.Rope(torch.from_numpy(f).cuda()), pos=torch.from_numpy(pos).cuda().reshape(1, T), ws=ws)
    angle = np.array([[exact_angle(p, y) for y in f] for p in pos])
    want = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    e = 2.0 ** -23 + 2 * ref.U32  # as in check_append, |a| + |b| = 1
    for got in (host(out)[:, 0], host(kp)[:, 0, 0]):
        assert np.all(np.abs(got - want) <= e + ref.HALF_STEP["f16"] * (np.abs(want) + e) + ref.TINY["f16"])


def test_append_without_rotation_copies_bits(q, cuda):
    # no rope: q_out and the cache hold the inputs' bits, infinities and NaN too; seq None is the token's number
    import torch
    T, n_q, n_kv, D, page = 4, 2, 1, 64, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, n_q + 2 * n_kv, D), generator=g, device="cuda").to(torch.float16)
    x[1, :, 3], x[2, :, 5], x[3, :, 7] = math.inf, -math.inf, NAN
    kp = torch.zeros((T, n_kv, page, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    kc = q.KVCache(kp, vp)
    ws = q.attn_workspace(kc, n_q, 1)
    out = torch.zeros((T, n_q, D), dtype=torch.float16, device="cuda")
    table = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).reshape(T, 1).contiguous()
    kv_pos = torch.tensor([0, 7, 3, 1], dtype=torch.int32, device="cuda")
    q.attn_kv_append(kc, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], table, kv_pos, out, ws=ws)
    assert torch.equal(out.view(torch.int16), x[:, :n_q].contiguous().view(torch.int16))
    for t in range(T):
        for pages, head in ((kp, n_q), (vp, n_q + 1)):
            assert torch.equal(pages[T - 1 - t, 0, kv_pos[t]].view(torch.int16), x[t, head].view(torch.int16))
    # q in place, then keys alone (no queries)
    y = x.clone()
    rope = q.Rope(torch.rand(32, device="cuda"))
    pos = torch.tensor([[5, 6, 7, 8]], dtype=torch.int32, device="cuda")
    q.attn_kv_append(kc, x[:, :n_q], x[:, n_q:n_q + 1], x[:, n_q + 1:], table, kv_pos, out, rope=rope, pos=pos, ws=ws)
    k_ref = kp.clone()
    q.attn_kv_append(kc, y[:, :n_q], y[:, n_q:n_q + 1], y[:, n_q + 1:], table, kv_pos, y[:, :n_q], rope=rope, pos=pos, ws=ws)
    assert torch.equal(y[:, :n_q].contiguous().view(torch.int16), out.view(torch.int16))
    assert torch.equal(y[:, n_q:].contiguous().view(torch.int16), x[:, n_q:].contiguous().view(torch.int16))
    q.attn_kv_append(kc, None, x[:, n_q:n_q + 1], x[:, n_q + 1:], table, kv_pos, rope=rope, pos=pos, ws=ws)
    assert torch.equal(kp.view(torch.int16), k_ref.view(torch.int16))
    assert q.qe_workspace_status(ws) == q.QE_OK


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_elements_past_the_rotation_keep_their_bits(q, cuda, adjacent, dtype):
    # every rotary_dim of a head: what lies behind it is copied, with a NaN's payload
    import torch
    T, D = 2, 128
    kp = torch.zeros((T, 1, 8, D), dtype=dt(dtype), device="cuda")
    kc = q.KVCache(kp, torch.zeros_like(kp))
    ws = q.attn_workspace(kc, 1, 1)
    table = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    exponent = {"f16": 0x7c00, "bf16": 0x7f80}[dtype]
    bits = torch.arange(T * D, device="cuda").remainder(60).add(1 + exponent).to(torch.int16)
    x = torch.where(torch.arange(T * D, device="cuda") % 2 == 0, bits, bits - 32768).to(torch.int16).view(dt(dtype)).reshape(T, 1, D)
    assert bool(x.isnan().all())
    for rd in range(0, D + 1, 16):
        out = torch.zeros((T, 1, D), dtype=dt(dtype), device="cuda")
        rope = q.Rope(torch.rand(rd // 2, device="cuda"), adjacent=adjacent)
        q.attn_kv_append(kc, x, x, x, table, at, out, rope=rope, ws=ws)
        for got in (out[:, :, rd:], kp[:, :, 0, rd:]):
            assert torch.equal(got.contiguous().view(torch.int16), x[:, :, rd:].contiguous().view(torch.int16)), rd
        assert bool(out[:, :, :rd].isnan().all())


def test_append_records_bad_places_and_writes_nothing_there(q, cuda):
    import torch
    T, D, page = 5, 64, 8
    x = torch.ones((T, 3, D), dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros((3, 1, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kc = q.KVCache(kp, vp)
    ws = q.attn_workspace(kc, 1, 1)
    out = torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 3], [-1, 1]], dtype=torch.int32, device="cuda")
    for seq, at in ((0, 8), (1, 0), (0, 16), (2, 0), (-1, 0)):  # page 3 of 3; page -1; column 2 of 2; sequence 2 of 2
        s = torch.zeros(T, dtype=torch.int32, device="cuda")
        p = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        s[3], p[3] = seq, at
        s[1], p[1] = 1, 9  # a good one beside it
        out.zero_()
        kp.zero_()
        q.attn_kv_append(kc, x[:, :1], x[:, 1:2], x[:, 2:], table, p, out, seq=s, ws=ws)
        assert q.qe_workspace_status(ws) == q.QE_ERR_INVALID_ARG
        assert q.qe_workspace_status(ws) == q.QE_OK
        assert bool((out[3] == 1).all()) and bool((out[1] == 1).all()) and bool((out[[0, 2, 4]] == 0).all())
        assert float(kp.float().sum()) == D and bool((kp[1, 0, 1] == 1).all())


# ---------------------------------------------------------------- attention

def attend_inputs(dtype, D, n_kv, G, page, prefix, lens, seed=0, cols=None, gap=0, scale_q=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed)
    B = len(lens)
    n_pre = -(-prefix // page)
    cols = cols or max(1, max(-(-max(n, 0) // page) for n in lens))
    n_pages = n_pre + B * cols + 2
    order = rng.permutation(n_pages).astype(np.int32)
    d = dict(B=B, dtype=dtype, D=D, n_kv=n_kv, G=G, page=page, prefix=prefix, lens=list(lens))
    d["pp"], d["tb"] = order[:n_pre], order[n_pre:n_pre + B * cols].reshape(B, cols).copy()
    for n in ("kp", "vp"):
        pool = torch.full((n_pages, n_kv * page * D + gap), NAN, device="cuda", dtype=dt(dtype))
        d[n] = pool[:, :n_kv * page * D].unflatten(1, (n_kv, page, D))
        full = torch.randn((n_pages, n_kv, page, D), generator=g, device="cuda").to(dt(dtype))
        # what no row may read stays NaN: the ends of last pages, unused pages
        used = np.zeros(n_pages, np.int64)
        used[order[:n_pre]] = np.clip(prefix - page * np.arange(n_pre), 0, page)
        used[d["tb"]] = np.clip(np.maximum(np.array(lens), 0)[:, None] - page * np.arange(cols)[None, :], 0, page)
        there = torch.from_numpy(np.arange(page)[None, :] < used[:, None]).cuda()[:, None, :, None]
        d[n].copy_(torch.where(there, full, NAN))
    d["q"] = (scale_q * torch.randn((B, n_kv * G, D), generator=g, device="cuda")).to(dt(dtype))
    d["scale"] = 1.3 / math.sqrt(D)
    return d


def run_attend(q, d, ws=None, out=None, stream=None):
    import torch
    kc = q.KVCache(d["kp"], d["vp"])
    n_q = d["n_kv"] * d["G"]
    ws = ws if ws is not None else q.attn_workspace(kc, n_q, d["B"])
    out = out if out is not None else torch.full((d["B"], n_q, d["D"]), 7.0, device="cuda").to(dt(d["dtype"]))
    lse = torch.full((d["B"], n_q), 7.0, device="cuda")
    q.attn_decode_step(kc, d["q"], out, torch.from_numpy(d["tb"]).cuda(),
                       torch.tensor(d["lens"], dtype=torch.int32, device="cuda"),
                       torch.from_numpy(d["pp"]).cuda() if d["prefix"] else None, d["prefix"], d["scale"], lse, ws, stream)
    return out, lse, ws


def check_attend(d, out, lse, rows=None, skip_keys=()):
    kp, vp, qq = host(d["kp"]), host(d["vp"]), host(d["q"])
    out, lse = host(out), lse.double().cpu().numpy()
    G = d["G"]
    for b in rows if rows is not None else range(d["B"]):
        if d["lens"][b] < 0:
            assert np.all(out[b] == 7.0) and np.all(lse[b] == 7.0)
            continue
        for h in range(d["n_kv"]):
            k, v = (np.concatenate([ref.gather(p, d["page"], d["pp"], d["prefix"], h),
                                    ref.gather(p, d["page"], d["tb"][b], d["lens"][b], h)]) for p in (kp, vp))
            keep = [j for j in range(len(k)) if (b, j) not in skip_keys]
            sl = slice(h * G, (h + 1) * G)
            want, want_lse, tol, tol_lse = ref.attend(qq[b, sl], k[keep], v[keep], d["scale"], d["dtype"])
            bad = np.abs(out[b, sl] - want) - tol
            assert np.all(bad <= 0), (b, h, bad.max())
            with np.errstate(invalid="ignore"):
                ok = (lse[b, sl] == want_lse) | (np.abs(lse[b, sl] - want_lse) <= tol_lse)
            assert ok.all(), (b, h, lse[b, sl], want_lse)


ATTEND = [
    # dtype, D, n_kv, G, page, prefix, lens
    ("bf16", 128, 2, 4, 16, 0, [1]),
    ("f16", 128, 1, 1, 16, 0, [0, 1, 15, 16, 17, 63, 64, 65]),
    ("bf16", 64, 2, 5, 1, 0, [33, 0, 129]),
    ("f16", 256, 1, 16, 24, 70, [0, 1, 200]),
    ("bf16", 128, 3, 7, 5, 1, [0, 0, 3]),
    ("f16", 64, 1, 17, 64, 64, [10, 300]),
    ("bf16", 128, 2, 40, 32, 65, [5, -1, 64]),
    ("bf16", 256, 2, 2, 128, 127, [1] * 9),
    ("f16", 128, 4, 8, 16, 300, [7, 0, -1, 90, 1000, 2, 31, 32, 33, 4, 5]),
    ("bf16", 64, 1, 3, 48, 513, [11 * i for i in range(50)]),
    ("f16", 128, 1, 1, 16, 130, [3] * 70),
    ("bf16", 128, 8, 4, 16, 1000, [i % 5 for i in range(33)]),
    ("f16", 64, 2, 4, 8, 2049, [17] * 40),
    ("bf16", 256, 1, 8, 64, 700, [9, 0, 100] * 11),
    ("bf16", 128, 1, 1, 16, 0, [3000]),
    # several blocks and tiles for each multiprocessor: own rows, one row a block and large groups
    ("f16", 64, 4, 2, 16, 0, [(37 * i) % 700 for i in range(100)]),
    ("bf16", 128, 8, 3, 32, 0, [(97 * i) % 500 for i in range(90)]),
    ("f16", 256, 4, 4, 64, 0, [(61 * i) % 400 for i in range(90)]),
    ("bf16", 64, 1, 70, 16, 10, [900, 0, 40]),
    ("f16", 128, 1, 300, 16, 0, [5, 2000]),
    ("bf16", 256, 1, 130, 16, 200, [700, 300]),
    # prefixes of many tiles, 65 to 300 rows
    ("f16", 64, 2, 4, 64, 20000, [(13 * i) % 90 for i in range(70)]),
    ("bf16", 128, 2, 4, 64, 20000, [(13 * i) % 90 for i in range(70)]),
    ("bf16", 128, 8, 2, 64, 9000, [3] * 40),
    ("f16", 256, 2, 4, 64, 20000, [(13 * i) % 90 for i in range(33)]),
    ("bf16", 64, 1, 1, 64, 40000, [200] * 66),
    # more blocks of the prefix's rows than multiprocessors
    ("f16", 64, 1, 16, 16, 200, [1] * 2600),
]


@pytest.mark.parametrize("c", ATTEND, ids=lambda c: f"{c[0]}_d{c[1]}_kv{c[2]}_g{c[3]}_page{c[4]}_pre{c[5]}_b{len(c[6])}")
def test_attention_matches_the_definition(q, cuda, c):
    d = attend_inputs(*c, seed=1)
    out, lse, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_OK
    check_attend(d, out, lse)
    again, lse2, _ = run_attend(q, d, ws=ws)  # the same workspace, the same bits
    import torch
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_peaked_scores_and_page_gaps(q, cuda):
    # scores of hundreds (one key takes all), pages apart in a larger pool
    for prefix, lens in ((0, [200, 9]), (150, [40] * 20)):
        d = attend_inputs("bf16", 128, 2, 4, 16, prefix, lens, seed=2, gap=4096, scale_q=60.0)
        out, lse, _ = run_attend(q, d)
        check_attend(d, out, lse)


@pytest.mark.parametrize("scale", [0.0, 1e-45, 2.0 ** -140], ids=["0", "smallest", "subnormal"])
@pytest.mark.parametrize("c", [("bf16", 128, 1, 4, 16, 300, [7, 0, 130] * 15), ("f16", 64, 1, 300, 16, 0, [5, 200]),
                               ("bf16", 256, 1, 8, 64, 70, [9] * 20), ("f16", 128, 2, 4, 16, 33, [5, 0, 64])],
                         ids=["wide", "wide_own", "d256", "narrow"])
def test_a_scale_of_zero_gives_the_mean(q, cuda, c, scale):
    d = dict(attend_inputs(*c, seed=17), scale=scale)
    out, lse, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_OK
    check_attend(d, out, lse)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 19 / 3, 1e9, 2.0 ** 64], ids=["1", "2e5", "1e9", "2^64"])
@pytest.mark.parametrize("dtype,D,B,G,prefix,n", [("f16", 128, 70, 4, 300, 40), ("bf16", 64, 2, 4, 0, 700),
                                                  ("f16", 256, 3, 2, 130, 5), ("bf16", 256, 40, 4, 300, 9)])
def test_scores_beyond_the_mantissa(q, cuda, dtype, D, B, G, prefix, n, scale):
    """Whole numbers as q and k: their products' sums are exact, and two sums differ by 1 at
    least.  From a scale of 1e5 on every weight but the largest sum's is 0: out is the mean of
    the values that have it."""
    import torch
    d = attend_inputs(dtype, D, 1, G, 16, prefix, [n] * B, seed=18)
    g = torch.Generator(device="cuda").manual_seed(19)
    for name in ("kp", "vp"):
        d[name] = torch.randint(-9, 10, d[name].shape, generator=g, device="cuda").to(dt(dtype))
    d["q"] = torch.randint(-9, 10, d["q"].shape, generator=g, device="cuda").to(dt(dtype))
    d["scale"] = scale
    out, lse, _ = run_attend(q, d)
    if scale == 1.0:
        return check_attend(d, out, lse)
    kp, vp, qq, out, lse = (host(x) for x in (d["kp"], d["vp"], d["q"], out, lse))
    for b in range(B):
        k, v = (np.concatenate([ref.gather(p, 16, d["pp"], prefix, 0), ref.gather(p, 16, d["tb"][b], n, 0)]) for p in (kp, vp))
        s = qq[b] @ k.T
        best = s == s.max(axis=1, keepdims=True)
        want = (best @ v) / best.sum(axis=1, keepdims=True)
        # l and the sums of values are small whole numbers; 1 / l, the product and the result are rounded
        assert np.all(np.abs(out[b] - want) <= (ref.HALF_STEP[dtype] + 2.0 ** -22) * np.abs(want))
        # scale log2(e), its product with the score, the logarithm's sum and the product with ln 2
        want = np.float64(np.float32(scale)) * s.max(axis=1) + np.log(best.sum(axis=1))
        assert np.all(np.abs(lse[b] - want) <= 6 * ref.U32 * np.abs(want))


@pytest.mark.parametrize("G,prefix,n", [(1, 0, 60000), (64, 30000, 0)], ids=["own_keys", "prefix"])
def test_fp16_keeps_the_tail_of_long_rows(q, cuda, G, prefix, n):
    """One key of weight 1 and value 0, all others of weight 2^-25.5 and value 1000, in segments that
    begin with the one: fp16 numerators that have 2^0 for the largest would lose every other."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = sms if not prefix else 4 * sms  # a row of own keys, or a block of 256 prefix rows, for each multiprocessor
    d = attend_inputs("f16", 64, 1, G, 64, prefix, [n], seed=20)
    d["B"], d["lens"], d["tb"] = B, [n] * B, np.repeat(d["tb"], B, axis=0)
    d["q"] = torch.zeros((B, G, 64), dtype=torch.float16, device="cuda")
    d["q"][:, :, 3] = 1.0
    tail = -17.6875
    d["kp"][:, :, :, :] = 0.0
    d["kp"][:, :, :, 3] = tail
    d["vp"][:, :, :, :] = 1000.0
    at = (d["pp"] if prefix else d["tb"][0])[0]
    d["kp"][at, 0, 0, 3], d["vp"][at, 0, 0] = 0.0, 0.0
    d["scale"] = 1.0
    out, lse, _ = run_attend(q, d)
    keys = prefix + n
    w = math.exp(tail)
    total = 1 + (keys - 1) * w
    want = 1000.0 * (keys - 1) * w / total
    # a numerator is off by 2^-25 (half of fp16's smallest) where the largest is 2^7, the sums by
    # their terms' roundings, the result by half a step
    tol = 1000.0 * keys * 2.0 ** -32 / total + (keys + 64) * 2 * ref.U32 * want + ref.HALF_STEP["f16"] * want
    assert tol < want / 20
    assert np.abs(host(out) - want).max() <= tol
    assert np.abs(host(lse) - math.log(total)).max() <= (keys + 64) * 2 * ref.U32 + 2.0 ** -21


def test_strided_queries_and_outputs(q, cuda):
    import torch
    d = attend_inputs("f16", 64, 2, 2, 16, 20, [30, 5, 70], seed=3)
    dense, lse, _ = run_attend(q, d)
    wide = torch.zeros((3, 8, 64), dtype=torch.float16, device="cuda")
    wide[:, 2:6] = d["q"]
    d2 = dict(d, q=wide[:, 2:6])
    into = torch.zeros((3, 12, 64), dtype=torch.float16, device="cuda")
    out, _, _ = run_attend(q, d2, out=into[:, 4:8])
    assert torch.equal(out, dense)
    assert bool((into[:, :4] == 0).all()) and bool((into[:, 8:] == 0).all())


def test_places_of_the_same_rows(q, cuda):
    # q, k, v, q_out and the attention's out as slices of one buffer's rows; q in place beside k and v
    import torch
    T, n_q, n_kv, D, page = 9, 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(24)
    first = torch.randn((T, 3 * n_q + 2 * n_kv, D), generator=g, device="cuda").to(torch.bfloat16)
    kp = torch.zeros((T, n_kv, page, D), dtype=torch.bfloat16, device="cuda")
    kc = q.KVCache(kp, torch.zeros_like(kp))
    ws = q.attn_workspace(kc, n_q, T)
    table = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    rope = q.Rope(torch.rand(D // 2, generator=g, device="cuda"))
    pos = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")

    def step(x, to, out):
        q.attn_kv_append(kc, x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:n_q + 2 * n_kv], table, at, to, rope=rope,
                         pos=pos, ws=ws)
        q.attn_decode_step(kc, to, out, table, at + 1, ws=ws)
        return to.clone(), out.clone(), kp.clone()

    new = torch.zeros((2, T, n_q, D), dtype=torch.bfloat16, device="cuda")
    want = step(first, new[0], new[1])
    x = first.clone()
    got = step(x, x[:, -n_q:], x[:, n_q + 2 * n_kv:-n_q])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(x[:, :n_q + 2 * n_kv], first[:, :n_q + 2 * n_kv])
    x = first.clone()
    got = step(x, x[:, :n_q], x[:, -n_q:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(x[:, n_q:-n_q], first[:, n_q:-n_q])
    assert q.qe_workspace_status(ws) == q.QE_OK


@pytest.mark.parametrize("T", [5, 3000])
def test_what_padding_rows_hold_does_not_matter(q, cuda, T):
    # padding rows of NaN, with positions, sequences and lengths out of any range: the others' results, bit for bit
    import torch
    n_q, n_kv, D, page = 4, 2, 64, 8
    g = torch.Generator(device="cuda").manual_seed(25)
    x = torch.randn((T, n_q + 2 * n_kv, D), generator=g, device="cuda").to(torch.bfloat16)
    pad = torch.arange(T, device="cuda") % 3 == 1
    rope = q.Rope(torch.rand(D // 2, generator=g, device="cuda"))
    table = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    got = []
    for filled in (False, True):
        y, kv_pos = x.clone(), torch.full((T,), 3, dtype=torch.int32, device="cuda")
        pos, seq = kv_pos + 100, torch.arange(T, dtype=torch.int32, device="cuda")
        kv_pos[pad] = -1
        if filled:
            y[pad] = NAN
            kv_pos[pad], pos[pad], seq[pad] = -2147483648, 2147483647, 2147483647
        kp = torch.zeros((T, n_kv, page, D), dtype=torch.bfloat16, device="cuda")
        kc = q.KVCache(kp, torch.zeros_like(kp))
        out, o = torch.full((2, T, n_q, D), 5.0, dtype=torch.bfloat16, device="cuda")
        ws = q.attn_workspace(kc, n_q, T)
        q.attn_kv_append(kc, y[:, :n_q], y[:, n_q:n_q + n_kv], y[:, n_q + n_kv:], table, kv_pos, out, rope=rope, pos=pos,
                         seq=seq, ws=ws)
        lens = torch.where(pad, kv_pos, 4)
        pp = torch.zeros(1, dtype=torch.int32, device="cuda")
        q.attn_decode_step(kc, y[:, :n_q], o, table, lens, pp, 4, ws=ws)  # the prefix's blocks hold all rows
        assert q.qe_workspace_status(ws) == q.QE_OK
        assert bool((out[pad] == 5).all()) and bool((o[pad] == 5).all())
        got.append((out, o, kc.k, kc.v))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not bool(got[0][1].isnan().any())


def test_bad_pages_are_masked_and_recorded(q, cuda):
    d = attend_inputs("bf16", 64, 1, 4, 8, 24, [20, 40], seed=4)
    good = d["tb"][1, 2]
    d["tb"][1, 2] = len(d["kp"])       # keys 16 .. 23 of row 1
    out, lse, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_ERR_INVALID_ARG
    d["tb"][1, 2] = good
    check_attend(d, out, lse, skip_keys={(1, 24 + j) for j in range(16, 24)})
    d["pp"][1] = -1                    # keys 8 .. 15 of the prefix, for both rows
    keep = d["pp"].copy()
    out, lse, _ = run_attend(q, d, ws=ws)
    assert q.qe_workspace_status(ws) == q.QE_ERR_INVALID_ARG
    d["pp"][1] = d["pp"][0]
    check_attend(d, out, lse, skip_keys={(b, j) for b in range(2) for j in range(8, 16)})
    d["pp"] = keep


def test_length_beyond_the_table_is_cut(q, cuda):
    d = attend_inputs("f16", 64, 1, 2, 8, 0, [16, 16], seed=5)
    d["lens"] = [16, 17]
    out, lse, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_ERR_INVALID_ARG
    d["lens"] = [16, 16]
    check_attend(d, out, lse)


def test_no_table_at_all(q, cuda):
    # table with no columns: every row has the prefix alone
    import torch
    d = attend_inputs("bf16", 128, 1, 4, 16, 100, [0, 0, 0], seed=6)
    full, lse, _ = run_attend(q, d)
    d["tb"] = np.zeros((3, 0), np.int32)
    out, lse2, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_OK
    assert torch.equal(out, full) and torch.equal(lse, lse2)
    check_attend(d, out, lse)


def test_a_nan_row_stays_alone(q, cuda):
    # NaN in one query: that row's heads are NaN, the others untouched by it
    import torch
    d = attend_inputs("bf16", 64, 2, 4, 16, 200, [5, 6, 7, 8, 9, 10], seed=7)
    clean, _, _ = run_attend(q, d)
    d["q"][2, 1, 0] = NAN
    out, lse, _ = run_attend(q, d)
    assert bool(out[2, 1].isnan().all()) and bool(lse[2, 1].isnan())
    keep = torch.ones((6, 8), dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(out[keep], clean[keep])


def test_offsets_beyond_32_bits(q, cuda):
    # pages 2^31 elements apart: byte offsets pass 2^32, element offsets 2^31
    import torch
    stride = (1 << 30) + 4096
    pool = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda")
    d = attend_inputs("bf16", 64, 1, 2, 16, 16, [13], seed=8)
    small, lse, _ = run_attend(q, d)
    far = {}
    for n, base in (("kp", 0), ("vp", 8192)):
        far[n] = torch.as_strided(pool, (3, 1, 16, 64), (stride, 1024, 64, 1), base)
        far[n][2] = d[n][d["pp"][0]]
        far[n][1] = d[n][d["tb"][0, 0]]
    d2 = dict(d, kp=far["kp"], vp=far["vp"], pp=np.array([2], np.int32), tb=np.array([[1]], np.int32))
    out, lse2, ws = run_attend(q, d2)
    assert torch.equal(out, small) and torch.equal(lse, lse2)
    # and the append reaches them
    kc = q.KVCache(far["kp"], far["vp"])
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    one = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    q.attn_kv_append(kc, None, x, 2 * x, one, torch.tensor([15], dtype=torch.int32, device="cuda"), ws=ws)
    assert bool((far["kp"][2, 0, 15] == 1).all()) and bool((far["vp"][2, 0, 15] == 2).all())
    del pool, far


def test_rows_of_one_sequence_give_a_causal_block(q, cuda):
    # several query tokens of one sequence: rows with the same pages, lengths one apart
    d = attend_inputs("f16", 128, 2, 2, 16, 40, [10, 11, 12, 13], seed=9)
    d["tb"][:] = d["tb"][3]
    out, lse, _ = run_attend(q, d)
    check_attend(d, out, lse)


def test_graphs_sharing_a_workspace_follow_new_lengths(q, cuda):
    # two captured calls on one workspace, replayed in turn; lengths change between replays
    import torch
    ds = [attend_inputs("bf16", 128, 2, 4, 16, 100, [50, 3, 90, 0], seed=10, cols=8),
          attend_inputs("f16", 64, 4, 2, 8, 0, [20, 64], seed=11, cols=8)]
    calls, ws = [], None
    for d in ds:
        kc = q.KVCache(d["kp"], d["vp"])
        n = q.attn_workspace_bytes(kc, d["n_kv"] * d["G"], d["B"])
        if ws is None or ws.numel() < n:
            ws = q.attn_workspace(kc, d["n_kv"] * d["G"], d["B"])
    s = torch.cuda.Stream()
    for d in ds:
        kc = q.KVCache(d["kp"], d["vp"])
        n_q = d["n_kv"] * d["G"]
        out = torch.full((d["B"], n_q, d["D"]), 7.0, device="cuda").to(dt(d["dtype"]))
        lse = torch.full((d["B"], n_q), 7.0, device="cuda")
        tb, pp = torch.from_numpy(d["tb"]).cuda(), torch.from_numpy(d["pp"]).cuda()
        ln = torch.tensor(d["lens"], dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            q.attn_decode_step(kc, d["q"], out, tb, ln, pp if d["prefix"] else None, d["prefix"], d["scale"], lse, ws)
        calls.append((g, out, lse, ln, tb, pp))  # a graph reads what it captured: all of it stays alive
    for trim in (0, 1, 2):
        for d, (g, out, lse, ln, *_) in zip(ds, calls):
            ln.copy_(torch.tensor([max(n - trim, 0) for n in d["lens"]], dtype=torch.int32))
        for _ in range(2):
            for g, *_ in calls:
                g.replay()
        torch.cuda.synchronize()
        for d, (g, out, lse, ln, *_) in zip(ds, calls):
            e = dict(d, lens=[max(n - trim, 0) for n in d["lens"]])
            check_attend(e, out, lse)
    assert q.qe_workspace_status(ws) == q.QE_OK


def test_another_stream(q, cuda):
    import torch
    d = attend_inputs("bf16", 128, 2, 4, 16, 300, [50, 3, 900], seed=12)
    want, lse, _ = run_attend(q, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, lse2, _ = run_attend(q, d)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, lse2)


def test_two_calls_at_once(q, cuda):
    """Two streams, each call with a workspace of its own: neither sees the other."""
    import torch
    a = attend_inputs("bf16", 128, 2, 4, 16, 300, [50, 3, 900], seed=12)
    b = attend_inputs("bf16", 64, 2, 8, 32, 0, [1, 700, 0, 129, 2000], seed=14)
    want = [run_attend(q, d)[:2] for d in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(8):
        for i, d in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(run_attend(q, d))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse, ws in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("D,G,prefix,lens", [
    (128, 64, 0, [130] * 600), (64, 16, 0, [200] * 900), (256, 32, 0, [70, 129] * 300), (128, 2, 4000, [0] * 900),
], ids=["64_rows", "16_rows", "d256", "prefix"])
def test_queries_that_arrive_after_the_keys(q, cuda, D, G, prefix, lens):
    """Many segments a multiprocessor whose keys lie in L2 (every row has the same pages) and whose
    queries come from memory: a product must not begin before its queries have landed."""
    import torch
    d = attend_inputs("bf16", D, 1, G, 16, prefix, lens[:2], seed=15)
    g = torch.Generator(device="cuda").manual_seed(16)
    d["B"], d["lens"] = len(lens), lens
    d["tb"] = np.repeat(d["tb"][-1:], len(lens), axis=0)
    kc = q.KVCache(d["kp"], d["vp"])
    ws = q.attn_workspace(kc, G, d["B"])
    cold = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")  # twice the L2 cache
    first = torch.randn((d["B"], G, D), generator=g, device="cuda").to(torch.bfloat16)
    want = {}
    for trial in range(12):
        d["q"] = first if trial % 2 == 0 else -first  # what an earlier segment left is never right
        cold.fill_(trial)
        out, lse, _ = run_attend(q, d, ws=ws)
        if trial < 2:
            want[trial] = out, lse
            check_attend(d, out, lse, rows=range(trial, d["B"], 37))
        else:
            assert torch.equal(out, want[trial % 2][0]) and torch.equal(lse, want[trial % 2][1])
    assert q.qe_workspace_status(ws) == q.QE_OK


def test_a_wait_that_gives_up_leaves_the_gpu_usable(q, cuda):
    # a limit of a microsecond, which waits for memory can pass: whatever such calls return, the status says
    # whether it counts, and the calls after them are right
    import torch
    ds = [attend_inputs("bf16", 128, 2, 4, 16, 3000, [700, 0, 90] * 20, seed=27),
          attend_inputs("f16", 256, 1, 16, 64, 500, [4000, 3], seed=28), attend_inputs("bf16", 64, 4, 4, 5, 0, [300] * 70, seed=29)]
    want = [run_attend(q, d) for d in ds]
    try:
        q.qe_set_wait_budget_ns(1000)
        for trial in range(5):
            for d, (out, lse, ws) in zip(ds, want):
                got, lse2, _ = run_attend(q, d, ws=ws)
                status = q.qe_workspace_status(ws)
                assert status in (q.QE_OK, q.QE_ERR_TIMEOUT)
                assert status != q.QE_OK or (torch.equal(got, out) and torch.equal(lse2, lse))
    finally:
        q.qe_set_wait_budget_ns(200_000_000)
    for d, (out, lse, ws) in zip(ds, want):
        got, lse2, _ = run_attend(q, d, ws=ws)
        assert q.qe_workspace_status(ws) == q.QE_OK
        assert torch.equal(got, out) and torch.equal(lse2, lse)


def test_segments_longer_than_the_limit(q, cuda):
    # 128 rows of head_dim 256 are one softmax group's: the other waits for all of a prefix of 90 tiles a
    # multiprocessor, some hundred microseconds, for its first own keys.  That is no reason to give up
    import torch
    d = attend_inputs("bf16", 256, 1, 8, 64, 640, [300, 1, 0, 129] * 4, seed=30)
    d["pp"], d["prefix"] = np.tile(d["pp"], 2700), 2700 * 640
    want, lse, ws = run_attend(q, d)
    assert q.qe_workspace_status(ws) == q.QE_OK
    try:
        q.qe_set_wait_budget_ns(20_000)
        got, lse2, _ = run_attend(q, d, ws=ws)
        assert q.qe_workspace_status(ws) == q.QE_OK
    finally:
        q.qe_set_wait_budget_ns(200_000_000)
    assert torch.equal(got, want) and torch.equal(lse2, lse)
    # the prefix's keys are 640 keys 2700 times: as those 640 with ln 2700 more in their scores
    kp, vp, qq = host(d["kp"]), host(d["vp"]), host(d["q"])
    for b in (0, 2, 7):
        k, v = (np.concatenate([ref.gather(p, 64, d["pp"], 640, 0), ref.gather(p, 64, d["tb"][b], d["lens"][b], 0)])
                for p in (kp, vp))
        s = d["scale"] * (qq[b] @ k.T)
        s[:, :640] += math.log(2700)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        o = p @ v / p.sum(axis=1, keepdims=True)
        # numerators' and results' roundings to bf16, and the score's and the sums' in fp32
        tol = (2 * ref.HALF_STEP["bf16"] + 2.0 ** -9) * (p @ np.abs(v)) / p.sum(axis=1, keepdims=True)
        assert np.all(np.abs(host(got)[b] - o) <= tol)


def test_empty_batch(q, cuda):
    import torch
    d = attend_inputs("bf16", 64, 1, 2, 16, 0, [3], seed=13)
    kc = q.KVCache(d["kp"], d["vp"])
    ws = q.attn_workspace(kc, 2, 0)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    q.attn_decode_step(kc, e, e.clone(), torch.empty((0, 1), dtype=torch.int32, device="cuda"),
                       torch.empty(0, dtype=torch.int32, device="cuda"), ws=ws)
    torch.cuda.synchronize()


def test_another_current_device_is_refused(q, cuda, monkeypatch):
    # one GPU is enough: the binding is told that the current device is the next one
    import torch
    from quantized_expert_matvec_b200 import _binding
    d = attend_inputs("bf16", 64, 1, 2, 16, 0, [3], seed=26)
    kc = q.KVCache(d["kp"], d["vp"])
    ws, at = q.attn_workspace(kc, 2, 1), torch.zeros(1, dtype=torch.int32, device="cuda")
    tb, k = torch.from_numpy(d["tb"]).cuda(), d["q"][:, :1]
    monkeypatch.setattr(_binding, "_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
        q.attn_workspace(kc, 2, 1)
    with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
        q.attn_kv_append(kc, None, k, k, tb, at, ws=ws)
    with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
        q.attn_decode_step(kc, d["q"], torch.empty_like(d["q"]), tb, at, ws=ws)
    with pytest.raises(ValueError, match="cuda:0, the current device is cuda:1"):
        q.token_sample(torch.zeros((1, 8), device="cuda"), torch.zeros(1, device="cuda"), at)


def test_transposed_arguments_are_refused(q, cuda):
    # as many elements as wanted, in another order
    import torch
    d = attend_inputs("bf16", 64, 1, 2, 16, 0, [3, 4, 5], seed=31)
    kc = q.KVCache(d["kp"], d["vp"])
    ws, at = q.attn_workspace(kc, 2, 3), torch.zeros(3, dtype=torch.int32, device="cuda")
    tb, k = torch.from_numpy(d["tb"]).cuda(), d["q"][:, :1]
    rope = q.Rope(torch.rand(32, device="cuda"), [0, 1] * 16)
    pos = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match=r"pos must be \[2, 3\]"):
        q.attn_kv_append(kc, None, k, k, tb, at, rope=rope, pos=pos.t().contiguous(), ws=ws)
    q.attn_kv_append(kc, None, k, k, tb, at, rope=rope, pos=pos, ws=ws)
    q.attn_kv_append(kc, None, k, k, tb, at, rope=rope, pos=pos.flatten(), ws=ws)
    lse, out = torch.zeros((3, 2), device="cuda"), torch.empty_like(d["q"])
    with pytest.raises(ValueError, match=r"lse must be \[3, 2\]"):
        q.attn_decode_step(kc, d["q"], out, tb, at + 1, lse=lse.t().contiguous(), ws=ws)
    q.attn_decode_step(kc, d["q"], out, tb, at + 1, lse=lse, ws=ws)
    assert q.qe_workspace_status(ws) == q.QE_OK


def test_binding_refuses_before_any_launch(q, cuda):
    import torch
    d = attend_inputs("bf16", 64, 1, 2, 16, 16, [3], seed=14)
    kc = q.KVCache(d["kp"], d["vp"])
    ws = q.attn_workspace(kc, 2, 1)
    tb, ln = torch.from_numpy(d["tb"]).cuda(), torch.tensor([3], dtype=torch.int32, device="cuda")
    out = torch.empty_like(d["q"])
    with pytest.raises(ValueError, match="out must be"):
        q.attn_decode_step(kc, d["q"], out.float(), tb, ln, ws=ws)
    with pytest.raises(ValueError, match="kv_len"):
        q.attn_decode_step(kc, d["q"], out, tb, ln.long(), ws=ws)
    with pytest.raises(ValueError, match="prefix_pages"):
        q.attn_decode_step(kc, d["q"], out, tb, ln, prefix_len=16, ws=ws)
    with pytest.raises(ValueError, match="heads"):
        q.attn_decode_step(kc, d["q"].transpose(1, 2).contiguous().transpose(1, 2), out, tb, ln, ws=ws)
    with pytest.raises(q.QEError, match="too small"):
        q.attn_decode_step(kc, d["q"], out, tb, ln, ws=ws[:512])
    with pytest.raises(q.QEError, match="overlaps"):
        q.attn_decode_step(kc, d["q"], d["q"], tb, ln, ws=ws)
    with pytest.raises(ValueError, match="pages of k"):
        q.KVCache(d["kp"].transpose(2, 3), d["vp"].transpose(2, 3))
