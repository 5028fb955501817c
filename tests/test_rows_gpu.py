"""GPU parity of the 8-bit activation path (add_rmsnorm, quantize_rows,
ternary_gemm_i8, ternary_swiglu_gate_up_i8) and of lora_add against the CPU
oracle in 64 bits.

Codes and integer probes must match bit for bit. Tolerances, with u = 2^-24:
* q_scale and the norm's factor: an fp32 sum of k squares in any order is
  within k u relative, its root within half of that, and the mean, the added
  epsilon, the root, the reciprocal and two products add one u each.
* h: that plus one fp16 rounding (2^-11 relative, 2^-25 below the normals).
* ternary_gemm_i8: the sum is exact and two products follow: 2 u (2.01 u with
  their cross term).
* lora_add: fp32 sums of k products for the inner values, 2^-22 of each for
  their two fp16 parts, an fp32 sum of 2 rank products, then three roundings.
"""
from __future__ import annotations

import sys

import numpy as np
import pytest

import oracle
import synth
from helpers import assert_within, swiglu_h_bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
NAN = float("nan")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def pbg(gpu):
    import packed_bit_gemv_amd as m

    m.lib()
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def host(t):
    return t.cpu().numpy()


def norm_case(seed, m, k):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float32)
    res = (rng.standard_normal((m, k)) * 4).astype(np.float32)
    res[:, :: max(1, k // 3)] *= 12
    return x, res, rng.uniform(0.5, 1.5, k).astype(np.float32)


def check_norm(got, ref, k, res_in=True):
    r, h, q, qs = got
    rr, hh, qq, ss = ref
    g = (k / 2 + 8) * U
    if r is not None:
        assert np.array_equal(host(r), rr)
    if h is not None:
        assert_within(host(h).astype(np.float64), hh, np.abs(hh) * (2.0 ** -11 + g) * 1.001 + 2.0 ** -25, "h")
    if q is not None:
        qn = host(q)
        assert qn.shape[1] == oracle.words_per_row(k) * 16
        assert np.array_equal(qn[:, :k], qq) and not qn[:, k:].any()
        assert_within(host(qs), ss, np.abs(ss) * g * 1.001, "q_scale")


NORM_SHAPES = [(1, 1), (1, 63), (3, 64), (1, 4096), (2, 4100), (5, 4097), (7, 12288), (700, 260), (1030, 1024), (2, 16384),
               (3, 16388), (2, 20001), (1, 131072), (2500, 8), (600, 4096)]


@pytest.mark.parametrize("m,k", NORM_SHAPES)
def test_add_rmsnorm(pbg, m, k):
    say(f"add_rmsnorm m={m} k={k}")
    x, res, w = norm_case(10 + m + k, m, k)
    ref = oracle.add_rmsnorm(x, w, 1e-6, res)
    xd, rd, wd = dev(x), dev(res), dev(w)
    check_norm(pbg.add_rmsnorm(xd, wd, 1e-6, residual=rd, want="hq"), ref, k)
    r, h, q, qs = pbg.add_rmsnorm(xd, wd, 1e-6, residual=rd)
    assert q is None and qs is None
    check_norm((r, h, None, None), ref, k)
    r, h, q, qs = pbg.add_rmsnorm(xd, wd, 1e-6, residual=rd, want="q")
    assert h is None
    check_norm((r, None, q, qs), ref, k)
    # without a residual
    ref0 = oracle.add_rmsnorm(x, w, 1e-5)
    r, h, q, qs = pbg.add_rmsnorm(xd, wd, 1e-5, want="hq")
    assert r is xd
    check_norm((None, h, q, qs), ref0, k)
    # in place, into the residual's buffer and into x's
    r1 = rd.clone()
    got = pbg.add_rmsnorm(xd, wd, 1e-6, residual=r1, residual_out=r1, want="hq")
    assert got[0] is r1
    check_norm(got, ref, k)
    x1 = xd.clone()
    check_norm(pbg.add_rmsnorm(x1, wd, 1e-6, residual=rd, residual_out=x1, want="hq"), ref, k)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_add_rmsnorm_offsets(pbg, off):
    """Buffers that are only element-aligned, rows behind the last one left as they were."""
    m, k = 3, 4096
    x, res, w = norm_case(5, m, k)

    def at(a):
        t = torch.zeros(a.size + 8, dtype=torch.float32, device="cuda:0")
        t[off:off + a.size] = dev(a.reshape(-1))
        return t[off:off + a.size].view(a.shape)

    h = torch.full((m * k + 16,), 7.0, dtype=torch.float16, device="cuda:0")
    q = torch.full(((m + 1), k), 9, dtype=torch.int8, device="cuda:0")
    qs = torch.full((m + 1,), 5.0, device="cuda:0")
    ro = torch.full((m * k + 8,), 3.0, device="cuda:0")
    got = pbg.add_rmsnorm(at(x), at(w), 1e-6, residual=at(res), residual_out=ro[off:off + m * k].view(m, k),
                          h=h[off:off + m * k].view(m, k), q=q[:m], q_scale=qs[:m])
    check_norm(got, oracle.add_rmsnorm(x, w, 1e-6, res), k)
    assert (h[:off] == 7).all() and (h[off + m * k:] == 7).all() and (q[m] == 9).all() and qs[m] == 5
    assert (ro[:off] == 3).all() and (ro[off + m * k:] == 3).all()


@pytest.mark.parametrize("k", [4096, 4100, 37])
def test_add_rmsnorm_odd_rows(pbg, k):
    """Rows of zeros, NaN, infinities, sums of squares past fp32, magnitudes near both ends."""
    x = np.random.default_rng(1).standard_normal((8, k)).astype(np.float32)
    x[0] = 0
    x[1, 5] = np.nan
    x[2, 7] = np.inf
    x[3] *= np.float32(1e25)
    x[4] *= np.float32(1e-36)
    x[5] *= np.float32(1e-25)
    x[6, 3] = 3e4
    w = np.ones(k, np.float32)
    _, h, q, qs = pbg.add_rmsnorm(dev(x), dev(w), 1e-6, want="hq")
    h, q, qs = host(h).astype(np.float64), host(q), host(qs)
    assert not q[:4].any() and qs[0] == 0 and np.isnan(qs[1:4]).all() and not q[4].any() and qs[4] == 0
    assert np.isnan(h[1]).all() and np.isnan(h[2]).all() and np.isnan(h[3]).all() and not h[0].any()
    ref = oracle.add_rmsnorm(x[5:], w, 1e-6)
    check_norm((None, torch.from_numpy(h[5:]), torch.from_numpy(q[5:]), torch.from_numpy(qs[5:])), ref, k)


@pytest.mark.parametrize("m,k", [(1, 1), (1, 31), (2, 4096), (33, 4100), (5, 4104), (2, 12288), (900, 520), (3, 16392), (1, 131072),
                                 (2, 40008), (2048, 8), (513, 12288)])
def test_quantize_rows(pbg, m, k):
    say(f"quantize_rows m={m} k={k}")
    x = (np.random.default_rng(m + k).standard_normal((m, k)) * 0.7).astype(np.float16)
    if m > 4:
        x[1] = 0
        x[2, k // 2] = np.nan
        x[3, 0] = -np.inf
        x[4] = np.float16(6e-8)
    qq, ss = oracle.quantize_rows(x)
    q, qs = pbg.quantize_rows(dev(x))
    qn = host(q)
    assert np.array_equal(qn[:, :k], qq) and not qn[:, k:].any()
    assert np.array_equal(host(qs), ss.astype(np.float32), equal_nan=True)
    # an element-aligned input
    t = torch.zeros(m * k + 3, dtype=torch.float16, device="cuda:0")
    t[3:] = dev(x).view(-1)
    q2, qs2 = pbg.quantize_rows(t[3:].view(m, k))
    assert torch.equal(q2, q) and np.array_equal(host(qs2), host(qs), equal_nan=True)


def pad(q):
    out = np.full((q.shape[0], 64 * ((q.shape[1] + 63) // 64)), 77, np.int8)  # readers ignore the padding
    out[:, :q.shape[1]] = q
    return out


GEMM_SHAPES = [(1, 1, 1), (1, 17, 64), (2, 5, 65), (16, 16, 256), (17, 33, 320), (1, 6144, 4096), (7, 4096, 12288), (8, 1024, 4096),
               (33, 100, 4100), (64, 48, 1000), (100, 1024, 4096), (129, 130, 192), (257, 300, 640), (300, 1000, 1096),
               (512, 512, 512), (1000, 257, 64), (2, 70000, 64), (70000, 3, 130), (130, 640, 12288), (513, 2050, 4096),
               (1, 9001, 200), (1, 50, 5000), (1, 5003, 5000), (1, 41, 9000), (1, 4201, 9000), (1, 30, 16384),
               (1, 4101, 16300), (1, 10, 20000), (2, 4097, 300), (2, 33, 8000), (2, 35, 12288), (2, 9, 14000),
               (3, 33, 4000), (4, 5001, 1000), (3, 8200, 100), (5, 300, 4096), (8, 2048, 70), (6, 100, 5000),
               (20, 9000, 700), (50, 900, 1100), (60, 4096, 300), (40, 6140, 600), (100, 4090, 500), (47, 12280, 260),
               (150, 4096, 900), (16, 16380, 300), (33, 2000, 257),  # and each tile, with rows, columns and K that end inside it
               (63, 12288, 580), (250, 12290, 328), (510, 12288, 700), (1000, 12290, 328)]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
def test_gemm_i8(pbg, m, n, k):
    say(f"gemm_i8 m={m} n={n} k={k}")
    rng = np.random.default_rng(m * 3 + n * 5 + k)
    q = rng.integers(-128, 128, (m, k)).astype(np.int8)
    codes = synth.ternary_codes(n + k, n, k)
    total = (torch.from_numpy(q).double() @ torch.from_numpy(codes).double().t()).numpy()
    packed = pbg.pack_ternary(dev(codes))[0]
    # powers of two as scales: exact
    s, qs = synth.pow2_scales(n, n), synth.pow2_scales(m + 1, m)
    buf = torch.full((m + 1, n), 5.0, device="cuda:0")
    y = pbg.ternary_gemm_i8(packed, dev(s), k, dev(pad(q)), dev(qs), buf[:m])
    assert np.array_equal(host(y).astype(np.float64), total * qs.astype(np.float64)[:, None] * s.astype(np.float64))
    assert (buf[m] == 5).all()
    # any scales: two roundings, NaN of a row without an 8-bit form stays in its row
    s, qs = synth.row_scales(n, n), synth.row_scales(m + 1, m)
    ref = total * qs.astype(np.float64)[:, None] * s.astype(np.float64)
    if m > 2:
        qs[1] = NAN
    y = host(pbg.ternary_gemm_i8(packed, dev(s), k, dev(pad(q)), dev(qs)))
    if m > 2:
        assert np.isnan(y[1]).all()
        y, ref = np.delete(y, 1, 0), np.delete(ref, 1, 0)
    assert_within(y, ref, np.abs(ref) * 2.01 * U, "gemm_i8")


def test_gemm_i8_largest_sum(pbg):
    """k at its limit, every product of the same sign: the int32 sums reach 2^30."""
    k = 131072
    codes = np.ones((3, k), np.int8)
    codes[1] = -1
    q = np.full((2, k), -128, np.int8)
    q[1] = 127
    one = np.ones(3, np.float32)
    y = host(pbg.ternary_gemm_i8(pbg.pack_ternary(dev(codes))[0], dev(one), k, dev(q), dev(one[:2])))
    assert np.array_equal(y, np.array([[-1, 1, -1], [0, 0, 0]]) * 128.0 * k + np.array([[0, 0, 0], [1, -1, 1]]) * 127.0 * k)


def test_gemm_i8_reads_every_code(pbg):
    """One nonzero activation at a time reads the packed codes back."""
    k, n = 200, 37
    codes = synth.ternary_codes(4, n, k)
    q = np.zeros((k, k), np.int8)
    np.fill_diagonal(q, 1)
    y = host(pbg.ternary_gemm_i8(pbg.pack_ternary(dev(codes))[0], dev(np.ones(n, np.float32)), k, dev(pad(q)),
                                 dev(np.ones(k, np.float32))))
    assert np.array_equal(y.T, codes)


def test_a_row_does_not_depend_on_its_batch(pbg):
    """The same bits for a row alone and among 2 to 600 others, whichever kernel takes them."""
    n, k, most = 520, 1088, 600
    rng = np.random.default_rng(9)
    q, qs = dev(rng.integers(-128, 128, (most, k)).astype(np.int8)), dev(synth.row_scales(1, most))
    w = [pbg.pack_ternary(dev(synth.ternary_codes(i, n, k)))[0] for i in (1, 2)]
    s = [dev(synth.row_scales(i, n)) for i in (3, 4)]
    y = pbg.ternary_gemm_i8(w[0], s[0], k, q, qs)
    h = pbg.ternary_swiglu_gate_up_i8(w[0], s[0], w[1], s[1], k, q, qs)
    for m in (1, 2, 3, 5, 8, 9, 17, 33, 64, 100, 257):
        a = slice(most - m, most)
        assert torch.equal(pbg.ternary_gemm_i8(w[0], s[0], k, q[a], qs[a]), y[a]), m
        assert torch.equal(pbg.ternary_swiglu_gate_up_i8(w[0], s[0], w[1], s[1], k, q[a], qs[a]), h[a]), m


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 12288, 4096), (8, 333, 4096), (16, 40, 72), (65, 100, 200), (130, 257, 1000),
                                   (300, 520, 4096), (40, 2048, 4096), (600, 130, 640), (30, 9000, 200), (63, 12300, 580),
                                   (20, 4000, 300), (40, 4090, 500), (47, 12280, 260), (9, 12288, 600), (1, 99, 5000), (1, 101, 9000), (1, 33, 16300), (1, 9, 20000), (2, 101, 500),
                                   (2, 50, 5000), (3, 40, 300),
                                   (100, 12290, 328), (256, 12300, 700), (510, 12290, 328)])
def test_swiglu_gate_up_i8(pbg, m, n, k):
    say(f"swiglu_gate_up_i8 m={m} n={n} k={k}")
    rng = np.random.default_rng(m + n + k)
    q = rng.integers(-128, 128, (m, k)).astype(np.int8)
    cg, cu = synth.ternary_codes(n + 1, n, k), synth.ternary_codes(n + 2, n, k)
    sg, su = synth.row_scales(3, n), synth.row_scales(4, n)
    qs = synth.row_scales(5, m) * np.float32(2 / np.sqrt(k))
    qd = torch.from_numpy(q).double()
    g = (qd @ torch.from_numpy(cg).double().t()).numpy() * qs.astype(np.float64)[:, None] * sg.astype(np.float64)
    u = (qd @ torch.from_numpy(cu).double().t()).numpy() * qs.astype(np.float64)[:, None] * su.astype(np.float64)
    buf = torch.full((m * n + 8,), 3.0, dtype=torch.float16, device="cuda:0")
    h = pbg.ternary_swiglu_gate_up_i8(pbg.pack_ternary(dev(cg))[0], dev(sg), pbg.pack_ternary(dev(cu))[0], dev(su), k,
                                      dev(pad(q)), dev(qs), buf[:m * n].view(m, n))
    sil = oracle.silu(g)
    assert_within(host(h).astype(np.float64), sil * u, swiglu_h_bound(sil, u, np.abs(g) * 2.01 * U, np.abs(u) * 2.01 * U), "h")
    assert (buf[m * n:] == 3).all()


def lora_case(seed, m, n, k, na, r, runs=False):
    rng = np.random.default_rng(seed)
    ids = rng.integers(-1, na + 1, m).astype(np.int32)  # -1 and na: no adapter
    if runs:
        ids.sort()
    return dict(y=rng.standard_normal((m, n)).astype(np.float32), x=rng.standard_normal((m, k)).astype(np.float16), ids=ids,
                a=(rng.standard_normal((na, r, k)) / np.sqrt(k)).astype(np.float16),
                b=(rng.standard_normal((na, n, r)) / np.sqrt(r)).astype(np.float16),
                scale=rng.uniform(0.5, 2, na).astype(np.float32))


def lora_bound(c):
    """Derived bound per element (see the module's docstring)."""
    na, r, k = c["a"].shape
    x, a, b, s = (np.abs(c[i].astype(np.float64)) for i in ("x", "a", "b", "scale"))
    out = np.abs(c["y"].astype(np.float64)) * U * 1.01
    for i, t in enumerate(c["ids"]):
        if 0 <= t < na:
            va = a[t] @ x[i]
            out[i] += s[t] * (b[t] @ va) * ((k + 16) * U + 2.0 ** -22 + 2 * r * U + 4 * U) * 1.01
    return out


LORA_SHAPES = [(1, 1, 1, 1, 1), (1, 4096, 4096, 4, 16), (5, 70, 64, 3, 8), (16, 33, 40, 20, 4), (64, 512, 4096, 24, 16),
               (40, 100, 100, 7, 12), (37, 260, 520, 2, 64), (100, 64, 264, 5, 128), (70, 200, 72, 70, 24), (300, 129, 640, 3, 32),
               (1000, 77, 130, 6, 16), (3, 50, 12288, 2, 16), (17, 6, 3, 2, 127), (600, 1100, 512, 4, 64)]


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("m,n,k,na,r", LORA_SHAPES)
def test_lora_add(pbg, m, n, k, na, r, runs):
    say(f"lora m={m} n={n} k={k} adapters={na} rank={r} runs={runs}")
    c = lora_case(m + n + k, m, n, k, na, r, runs)
    d = {i: dev(v) for i, v in c.items()}
    ref = oracle.lora_add(**c)
    buf = torch.full((m + 1, n), 5.0, device="cuda:0")
    ws = torch.full((pbg.lora_workspace(m, r, "cuda:0").numel() + 64,), 255, dtype=torch.uint8, device="cuda:0")  # any content
    out = pbg.lora_add(**d, out=buf[:m], workspace=ws)
    assert_within(host(out), ref, lora_bound(c), "lora")
    without = (c["ids"] < 0) | (c["ids"] >= na)
    assert np.array_equal(host(out)[without], c["y"][without]) and (buf[m] == 5).all()
    assert (ws[-64:] == 255).all()
    y = d["y"].clone()
    assert torch.equal(pbg.lora_add(**{**d, "y": y}, out=y), out)  # in place, the same bits


# Calls that put their rows in the order of the adapters first: more than one chunk of 4,096 rows, ids that share a
# bin (more than 1,023 adapters), odd ranks, few rows.
LORA_SORTED = [(1000, 1200, 1100, 100, 128), (4200, 300, 520, 1100, 17), (1531, 4100, 64, 64, 16), (130, 9000, 9000, 40, 64)]


@pytest.mark.parametrize("m,n,k,na,r", LORA_SORTED)
def test_lora_sorted(pbg, m, n, k, na, r):
    """Against the oracle; the order of the rows, and that of the sort's atomics, do not change a bit."""
    say(f"lora sorted m={m} n={n} k={k} adapters={na} rank={r}")
    c = lora_case(m + n + k, m, n, k, na, r)
    d = {i: dev(v) for i, v in c.items()}
    ws = torch.full((pbg.lora_workspace(m, r, "cuda:0").numel() + 64,), 255, dtype=torch.uint8, device="cuda:0")
    out = pbg.lora_add(**d, workspace=ws)
    assert_within(host(out), oracle.lora_add(**c), lora_bound(c), "lora")
    without = (c["ids"] < 0) | (c["ids"] >= na)
    assert np.array_equal(host(out)[without], c["y"][without])
    assert (ws[-64:] == 255).all()
    for _ in range(3):
        assert torch.equal(pbg.lora_add(**d, workspace=ws), out)
    by = torch.argsort(d["ids"], stable=True)
    runs = {**d, "y": d["y"][by].contiguous(), "x": d["x"][by].contiguous(), "ids": d["ids"][by].contiguous()}
    assert torch.equal(pbg.lora_add(**runs), out[by])
    one = {**d, "ids": torch.full_like(d["ids"], na - 1)}  # all rows in one bin
    assert_within(host(pbg.lora_add(**one)), oracle.lora_add(**{**c, "ids": host(one["ids"])}),
                  lora_bound({**c, "ids": host(one["ids"])}), "one adapter")
    assert torch.equal(pbg.lora_add(**{**d, "ids": torch.full_like(d["ids"], -1)}), d["y"])


def test_lora_sorted_graph(pbg):
    """Captured once, replayed on new ids and rows with eager work between: the eager result's bits every time."""
    m, n, k, na, r = 1531, 4100, 64, 64, 16
    d = {i: dev(v) for i, v in lora_case(1, m, n, k, na, r).items()}
    out, ws = torch.empty_like(d["y"]), pbg.lora_workspace(m, r, "cuda:0")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pbg.lora_add(**d, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pbg.lora_add(**d, out=out, workspace=ws)
    for i in range(4):
        c = lora_case(10 + i, m, n, k, na, r, runs=i == 2)
        for name in ("x", "y", "ids"):
            d[name].copy_(dev(c[name]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, pbg.lora_add(**d)), i


@pytest.mark.parametrize("m,k,r", [(3, 64, 8), (40, 192, 16), (300, 64, 64), (9, 60, 5)])
def test_lora_exact_probe(pbg, m, k, r):
    """Whole numbers and scales of powers of two: every sum is exact in fp32."""
    rng = np.random.default_rng(m)
    n, na = 50, 3
    c = dict(y=rng.integers(-99, 99, (m, n)).astype(np.float32), x=rng.integers(-8, 9, (m, k)).astype(np.float16),
             ids=rng.integers(-1, na, m).astype(np.int32), a=rng.integers(-3, 4, (na, r, k)).astype(np.float16),
             b=rng.integers(-3, 4, (na, n, r)).astype(np.float16), scale=np.array([0.5, 1, 2], np.float32))
    out = host(pbg.lora_add(**{i: dev(v) for i, v in c.items()}))
    assert np.array_equal(out.astype(np.float64), oracle.lora_add(**c))


def test_lora_other_adapters_stay_out(pbg):
    """NaN and infinities in one adapter reach only its own rows."""
    c = lora_case(2, 50, 96, 128, 4, 16)
    c["ids"][:] = np.arange(50) % 5 - 1
    ref = oracle.lora_add(**c)
    bound = lora_bound(c)
    c["a"][2], c["b"][2, 3:9] = np.nan, np.inf
    out = host(pbg.lora_add(**{i: dev(v) for i, v in c.items()}))
    ok = c["ids"] != 2
    assert_within(out[ok], ref[ok], bound[ok], "rows of other adapters")
    assert np.isnan(out[~ok]).any()


def test_lora_odd_offsets(pbg):
    """Element-aligned fp16 inputs take the guarded loads and give the same sums."""
    c = lora_case(8, 20, 64, 256, 3, 16)

    def at(v):
        if v.dtype != np.float16:
            return dev(v)
        t = torch.zeros(v.size + 1, dtype=torch.float16, device="cuda:0")
        t[1:] = dev(v).view(-1)
        return t[1:].view(v.shape)

    assert_within(host(pbg.lora_add(**{i: at(v) for i, v in c.items()})), oracle.lora_add(**c), lora_bound(c), "offsets")


def block(pbg, w, x, res, ids):
    """The feed-forward half of a layer on 8-bit rows with an adapter beside down, and the norm that follows."""
    r, _, q, qs = pbg.add_rmsnorm(x, w["norm"], 1e-6, residual=res, want="q")
    h = pbg.ternary_swiglu_gate_up_i8(w["gate"], w["sg"], w["up"], w["su"], w["d"], q, qs)
    hq, hs = pbg.quantize_rows(h)
    y = pbg.ternary_gemm_i8(w["down"], w["sd"], w["f"], hq, hs)
    pbg.lora_add(y, h, ids, w["a"], w["b"], w["s"], out=y)
    r2, h2, _, _ = pbg.add_rmsnorm(y, w["norm"], 1e-6, residual=r)
    return q, qs, h, hq, hs, y, r2, h2


def block_weights(pbg, d, f):
    rng = np.random.default_rng(d)
    cg, cu, cd = (synth.ternary_codes(i, f, d) for i in (1, 2)), None, synth.ternary_codes(3, d, f)
    cg, cu = cg
    np_w = dict(cg=cg, cu=cu, cd=cd, sg=synth.row_scales(4, f), su=synth.row_scales(5, f), sd=synth.row_scales(6, d),
                norm=rng.uniform(0.5, 1.5, d).astype(np.float32),
                a=(rng.standard_normal((3, 16, f)) / np.sqrt(f)).astype(np.float16),
                b=(rng.standard_normal((3, d, 16)) / 4).astype(np.float16), s=np.array([0.5, 1, 2], np.float32))
    w = {i: dev(v) for i, v in np_w.items() if not i.startswith("c")}
    w.update(gate=pbg.pack_ternary(dev(cg))[0], up=pbg.pack_ternary(dev(cu))[0], down=pbg.pack_ternary(dev(cd))[0], d=d, f=f)
    return np_w, w


@pytest.mark.parametrize("m", [1, 6, 200])
def test_block(pbg, m):
    """The operators together: each step against the oracle on the step's own inputs."""
    d, f = 256, 712
    nw, w = block_weights(pbg, d, f)
    x, res, _ = norm_case(m, m, d)
    ids = (np.arange(m) % 4 - 1).astype(np.int32)
    q, qs, h, hq, hs, y, r2, h2 = [host(t) for t in block(pbg, w, dev(x), dev(res), dev(ids))]
    r_ref, _, q_ref, qs_ref = oracle.add_rmsnorm(x, nw["norm"], 1e-6, res)
    assert np.array_equal(q[:, :d], q_ref)
    assert_within(qs, qs_ref, qs_ref * (d / 2 + 8) * U * 1.001, "q_scale")
    g = oracle.ternary_gemm_i8(oracle.pack(nw["cg"])[0], nw["sg"], d, q, qs)
    u = oracle.ternary_gemm_i8(oracle.pack(nw["cu"])[0], nw["su"], d, q, qs)
    sil = oracle.silu(g)
    assert_within(h.astype(np.float64), sil * u, swiglu_h_bound(sil, u, np.abs(g) * 2.01 * U, np.abs(u) * 2.01 * U), "h")
    assert np.array_equal(hq[:, :f], oracle.quantize_rows(h)[0])
    base = oracle.ternary_gemm_i8(oracle.pack(nw["cd"])[0], nw["sd"], f, hq, hs)
    c = dict(y=base, x=h, ids=ids, a=nw["a"], b=nw["b"], scale=nw["s"])
    assert_within(y, oracle.lora_add(**c), lora_bound(c) + np.abs(base) * 2.01 * U, "y")
    r_ref2, h_ref2, _, _ = oracle.add_rmsnorm(y, nw["norm"], 1e-6, r_ref)
    check_norm((torch.from_numpy(r2), torch.from_numpy(h2), None, None), (r_ref2, h_ref2, None, None), d)


def test_block_in_a_graph_and_on_a_stream(pbg):
    """Captured once and replayed on new inputs, with eager work between the replays; and on a side stream."""
    m, d, f = 5, 256, 712
    _, w = block_weights(pbg, d, f)
    x, res, ids = (torch.zeros((m, d), device="cuda:0"), torch.zeros((m, d), device="cuda:0"),
                   torch.zeros(m, dtype=torch.int32, device="cuda:0"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(pbg, w, x, res, ids)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(pbg, w, x, res, ids)
    for seed in range(4):
        xn, rn, _ = norm_case(seed, m, d)
        x.copy_(dev(xn))
        res.copy_(dev(rn))
        ids.copy_(dev((np.arange(m) + seed).astype(np.int32) % 4 - 1))
        graph.replay()
        torch.cuda.synchronize()
        eager = block(pbg, w, x, res, ids)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = block(pbg, w, x, res, ids)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b, c in zip(outs, eager, other):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_two_streams_at_once(pbg):
    """Two chains on two streams, separate workspaces: each keeps its results."""
    d, f = 256, 712
    _, w = block_weights(pbg, d, f)
    jobs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for m in (6, 90):
        x, res, _ = norm_case(m, m, d)
        a = dev(x), dev(res), dev((np.arange(m) % 4 - 1).astype(np.int32))
        jobs.append((a, block(pbg, w, *a)))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for (a, _), st in zip(jobs, streams):
            with torch.cuda.stream(st):
                outs.append(block(pbg, w, *a))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        for a, b in zip(got, jobs[i % 2][1]):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(pbg):
    """2^20 rows of 2,100 columns: element offsets past 2^31 in every operator, checked at rows across the range."""
    m, k, n = 1 << 20, 64, 2100
    some = np.array([0, 1, 511, 12345, m // 2 - 1, m // 2, m - 1000, m - 2, m - 1])
    at = torch.from_numpy(some).to("cuda:0")
    g = torch.Generator(device="cuda:0").manual_seed(1)
    q = torch.randint(-127, 128, (m, k), generator=g, device="cuda:0", dtype=torch.int8)
    qs = torch.rand(m, generator=g, device="cuda:0") + 0.5
    codes, s = synth.ternary_codes(5, n, k), synth.row_scales(6, n)
    y = pbg.ternary_gemm_i8(pbg.pack_ternary(dev(codes))[0], dev(s), k, q, qs)
    ref = oracle.ternary_gemm_i8(oracle.pack(codes)[0], s, k, host(q[at]), host(qs[at]))
    assert_within(host(y[at]), ref, np.abs(ref) * 2.01 * U, "y")
    w = np.ones(n, np.float32)
    r, h, hq, hs = pbg.add_rmsnorm(y, dev(w), 1e-6, want="hq")
    check_norm((None, h[at], hq[at], hs[at]), oracle.add_rmsnorm(host(y[at]), w, 1e-6), n)
    x2, xs2 = pbg.quantize_rows(h)
    rq, rs = oracle.quantize_rows(host(h[at]))
    assert np.array_equal(host(x2[at])[:, :n], rq) and np.array_equal(host(xs2[at]), rs.astype(np.float32))
    del hq, x2
    c = lora_case(3, len(some), n, n, 2, 8)
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda:0")
    ids[at] = dev(c["ids"] % 2)
    c.update(y=host(y[at]), x=host(h[at]), ids=host(ids[at]))
    out = pbg.lora_add(y, h, ids, dev(c["a"]), dev(c["b"]), dev(c["scale"]), out=y)
    assert_within(host(out[at]), oracle.lora_add(**c), lora_bound(c), "lora")


def test_refusals(pbg):
    x = torch.zeros((2, 64), device="cuda:0")
    w = torch.ones(64, device="cuda:0")
    h = x.half()
    with pytest.raises(pbg.PbgError):
        pbg.add_rmsnorm(x, w, 0.0)
    with pytest.raises(pbg.PbgError):
        pbg.add_rmsnorm(x[:0], w)
    for bad in (lambda: pbg.add_rmsnorm(h, w), lambda: pbg.add_rmsnorm(x, w[:63]), lambda: pbg.add_rmsnorm(x.t(), w),
                lambda: pbg.add_rmsnorm(x, w, residual=x[:1]), lambda: pbg.add_rmsnorm(x, w, want="x"),
                lambda: pbg.quantize_rows(x), lambda: pbg.quantize_rows(h, torch.zeros((2, 63), dtype=torch.int8, device="cuda:0")),
                lambda: pbg.ternary_gemm_i8(torch.zeros((4, 4), dtype=torch.int32, device="cuda:0"), torch.ones(4, device="cuda:0"),
                                            65, torch.zeros((2, 128), dtype=torch.int8, device="cuda:0"),
                                            torch.ones(2, device="cuda:0")),
                lambda: pbg.lora_add(x, h, torch.zeros(2, dtype=torch.int64, device="cuda:0"),
                                     torch.zeros((1, 8, 64), dtype=torch.float16, device="cuda:0"),
                                     torch.zeros((1, 64, 8), dtype=torch.float16, device="cuda:0"), torch.ones(1, device="cuda:0"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pbg.PbgError):
        pbg.lora_add(x, h, torch.zeros(2, dtype=torch.int32, device="cuda:0"),
                     torch.zeros((1, 8, 64), dtype=torch.float16, device="cuda:0"),
                     torch.zeros((1, 64, 8), dtype=torch.float16, device="cuda:0"), torch.ones(1, device="cuda:0"),
                     workspace=torch.zeros(16, dtype=torch.uint8, device="cuda:0"))


# ---- lora_add: the range of the inner values ---------------------------------

# Each form of the second launch: one block, the slices joined in it, the joining launch, 32 and 64 columns a wave, rows
# sorted by a launch before, odd ranks and widths.
LORA_WIDE = [(3, 24, 64, 2, 8), (9, 41, 60, 3, 5), (12, 300, 200, 3, 128), (40, 50, 192, 3, 16), (40, 70, 200, 3, 30),
             (300, 130, 64, 3, 64), (100, 300, 72, 4, 128), (1531, 4100, 72, 2, 64), (1000, 1200, 1100, 100, 128),
             (1531, 4101, 75, 40, 61)]


@pytest.mark.parametrize("span", [12, 36])
@pytest.mark.parametrize("m,n,k,na,r", LORA_WIDE)
def test_lora_inner_values_of_any_range(pbg, m, n, k, na, r, span):
    """Inner values of one row from 2^12 down to 2^(12 - span) of a whole number, each with its own rows of b: every sum
    has one term and every operation is exact, so each output is the small inner value itself, however large the others
    are. 12: two fp16 parts hold them; 36: they do not."""
    say(f"lora wide m={m} n={n} k={k} adapters={na} rank={r} span={span}")
    rng = np.random.default_rng(m + r)
    power = np.stack([rng.permutation(np.linspace(12, 12 - span, r).round()) for _ in range(na)])
    a = rng.integers(-3, 4, (na, r, k)) * 2.0 ** power[:, :, None]
    b = np.zeros((na, n, r), np.float16)
    rows = np.arange(n)
    b[:, rows, rows % r] = rng.choice([-3, -2, -1, 1, 2, 3], (na, n))
    c = dict(y=np.zeros((m, n), np.float32), x=rng.integers(-8, 9, (m, k)).astype(np.float16),
             ids=rng.integers(-1, na, m).astype(np.int32), a=a.astype(np.float16), b=b,
             scale=2.0 ** rng.integers(-1, 2, na).astype(np.float32))
    assert np.array_equal(c["a"].astype(np.float64), a)
    out = host(pbg.lora_add(**{i: dev(v) for i, v in c.items()}))
    assert np.array_equal(out.astype(np.float64), oracle.lora_add(**c))


@pytest.mark.parametrize("m,n,k,na,r", [(5, 70, 64, 3, 8), (40, 100, 100, 4, 12), (300, 129, 640, 4, 32), (100, 64, 264, 5, 128),
                                        (1531, 4100, 64, 64, 16)])
def test_lora_infinities(pbg, m, n, k, na, r):
    """An infinity in x, a, b or y reaches exactly the outputs that the formula gives it, with its sign; NaN only where
    the formula has one (infinities of both signs in a sum)."""
    say(f"lora infinities m={m} n={n} k={k} adapters={na} rank={r}")
    c = lora_case(m + n, m, n, k, na, r)
    c["ids"] = (np.arange(m) % (na + 1) - 1).astype(np.int32)
    for name in "xab":
        c[name][c[name] == 0] = 1
    c["a"][0, r // 2, 3] = np.inf           # every output of the rows of adapter 0
    c["b"][1, n // 2, r - 1] = -np.inf      # one output of the rows of adapter 1
    c["x"][3, 5] = -np.inf                  # a row of adapter 2
    c["x"][0, 7] = np.inf                   # a row without an adapter
    c["y"][2, 1] = np.inf                   # one output of a row of adapter 1
    with np.errstate(invalid="ignore"):
        ref, bound = oracle.lora_add(**c), lora_bound(c)
    out = host(pbg.lora_add(**{i: dev(v) for i, v in c.items()})).astype(np.float64)
    ok = np.isfinite(ref)
    assert np.isinf(ref[1]).all() and np.isinf(ref[2, n // 2]) and np.isinf(ref[2, 1]) and np.isnan(ref[3]).any() and ok[0].all()
    assert np.array_equal(out[~ok], ref[~ok], equal_nan=True)
    assert_within(out[ok], ref[ok], bound[ok], "finite outputs")


@pytest.mark.parametrize("m,n,k,na,r", [(5, 70, 64, 5, 8), (40, 100, 100, 5, 12), (300, 129, 640, 5, 32), (100, 64, 264, 5, 128)])
def test_lora_scales_of_any_size(pbg, m, n, k, na, r):
    """Scales of 0, below and near the smallest normal number and large ones, on small inner values: the product of the
    scale with the sum is the only rounding more, to half of 2^-149 below the normals."""
    say(f"lora scales m={m} n={n} k={k} rank={r}")
    c = lora_case(m + n, m, n, k, na, r)
    c["y"][:] = 0
    c["x"] = (c["x"] * np.float16(2.0 ** -8)).astype(np.float16)
    c["a"] = (c["a"] * np.float16(2.0 ** -6)).astype(np.float16)
    c["scale"] = np.array([0.0, 1.7 * 2.0 ** -130, 1.3 * 2.0 ** -120, -1.1 * 2.0 ** -100, 1.9 * 2.0 ** 110], np.float32)
    out = host(pbg.lora_add(**{i: dev(v) for i, v in c.items()}))
    assert_within(out, oracle.lora_add(**c), lora_bound(c) + 2.0 ** -149, "scales")


@pytest.mark.parametrize("r", [4, 16, 64])
def test_lora_one_workspace_for_fewer_rows(pbg, r):
    """A workspace allocated once for the most rows serves every smaller call, whatever it was used for before."""
    n, k, na = 80, 192, 3
    ws = pbg.lora_workspace(2100, r, "cuda:0")
    for m in (2100, 2048, 1000, 65, 64, 33, 28, 24, 17, 16, 15, 1):
        say(f"lora workspace rank={r} m={m}")
        mine = pbg.lora_workspace(m, r, "cuda:0")
        assert mine.numel() <= ws.numel()
        d = {i: dev(v) for i, v in lora_case(m + r, m, n, k, na, r).items()}
        assert torch.equal(pbg.lora_add(**d, workspace=ws), pbg.lora_add(**d, workspace=mine)), m
    ws = pbg.lora_workspace(17, r, "cuda:0")
    d = {i: dev(v) for i, v in lora_case(1, 16, n, k, na, r).items()}
    assert torch.equal(pbg.lora_add(**d, workspace=ws), pbg.lora_add(**d))


def test_a_row_does_not_depend_on_its_batch_in_any_tile(pbg):
    """The same bits for a row alone, in the streaming shapes and in every tile (from 33, 63, 100, 250, 510 and 1,000 rows
    on at this width), with an odd number of 64-column chunks."""
    n, k, most = 12290, 392, 1000
    rng = np.random.default_rng(19)
    q, qs = dev(pad(rng.integers(-128, 128, (most, k)).astype(np.int8))), dev(synth.row_scales(1, most))
    codes = [synth.ternary_codes(i, n, k) for i in (1, 2)]
    w = [pbg.pack_ternary(dev(c))[0] for c in codes]
    s = [dev(synth.row_scales(i, n)) for i in (3, 4)]
    y = pbg.ternary_gemm_i8(w[0], s[0], k, q, qs)
    h = pbg.ternary_swiglu_gate_up_i8(w[0], s[0], w[1], s[1], k, q, qs)
    ref = oracle.ternary_gemm_i8(oracle.pack(codes[0])[0], host(s[0]), k, host(q), host(qs))
    assert_within(host(y), ref, np.abs(ref) * 2.01 * U, "y")
    for m in (1, 2, 3, 8, 9, 17, 33, 63, 100, 160, 250, 400, 510, 700):
        say(f"same bits m={m}")
        a = slice(most - m, most)
        assert torch.equal(pbg.ternary_gemm_i8(w[0], s[0], k, q[a], qs[a]), y[a]), m
        assert torch.equal(pbg.ternary_swiglu_gate_up_i8(w[0], s[0], w[1], s[1], k, q[a], qs[a]), h[a]), m


@pytest.mark.parametrize("m,k", [(3, 1500), (1030, 1500), (1030, 2048), (1030, 3001), (1030, 4096)])
def test_add_rmsnorm_row_kernels(pbg, m, k):
    """The row kernels of 1,025 to 4,096 columns, for few and for many rows."""
    test_add_rmsnorm(pbg, m, k)


@pytest.mark.parametrize("m,k", [(1030, 3000), (1030, 5000), (1030, 12292), (1024, 16384), (3, 3000), (3, 5000)])
def test_quantize_rows_row_kernels(pbg, m, k):
    """The same for the quantizer, with rows of zeros, NaN and infinities."""
    test_quantize_rows(pbg, m, k)


# Every form of the launches at every padded rank, aligned and not: one block; 32 columns a wave; 64 from 384 workgroups
# on, with the last wave's columns cut.
LORA_FORMS = [(7, 70, 64, 2, 24), (7, 71, 65, 2, 25), (16, 100, 72, 2, 64), (16, 101, 75, 2, 41), (12, 130, 75, 2, 127),
              (300, 600, 72, 4, 16), (300, 500, 75, 3, 61),
              (1531, 4100, 72, 3, 16), (1531, 4100, 264, 3, 24), (1531, 4100, 72, 3, 64), (1531, 4100, 72, 4, 128),
              (1600, 4110, 75, 3, 13), (1531, 4099, 75, 3, 30), (1531, 4101, 75, 3, 61), (1531, 4099, 75, 3, 127)]


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("m,n,k,na,r", LORA_FORMS)
def test_lora_add_forms(pbg, m, n, k, na, r, runs):
    test_lora_add(pbg, m, n, k, na, r, runs)


LORA_SORTED_FORMS = [(1000, 2000, 4000, 60, 16), (1000, 2001, 4001, 60, 15), (1000, 2000, 1000, 60, 32),
                     (1000, 1001, 501, 60, 61), (1000, 600, 200, 60, 128), (1531, 4101, 75, 60, 13), (1531, 4100, 264, 30, 24),
                     (1531, 4099, 75, 60, 30), (1531, 4100, 72, 20, 64), (1531, 4101, 75, 20, 61), (1531, 4100, 72, 12, 128),
                     (1531, 4099, 75, 12, 127)]


@pytest.mark.parametrize("m,n,k,na,r", LORA_SORTED_FORMS)
def test_lora_sorted_forms(pbg, m, n, k, na, r):
    test_lora_sorted(pbg, m, n, k, na, r)


@pytest.mark.parametrize("m,n,k,na,r", [(16, 100, 72, 2, 64), (40, 100, 104, 3, 16), (300, 130, 72, 2, 24), (1531, 4100, 64, 64, 16)])
def test_lora_rows_do_not_share_their_range(pbg, m, n, k, na, r):
    """Rows of one group: some without inner values that two parts hold, some with infinities, NaN or zeros only. The
    other rows keep their bits."""
    say(f"lora neighbours m={m} n={n} k={k} adapters={na} rank={r}")
    c = lora_case(m + r, m, n, k, na, r)
    x = c["x"].copy()
    odd = np.arange(m) % 5 == 2
    x[odd] = np.float16(0)
    x[2::20, 0] = np.inf
    x[7::20, 0] = np.nan
    x[12::20, :] = np.float16(2.0 ** -24)
    x[12::20, 1] = np.float16(60000)
    c["a"][:, : r // 2, 1] = 0
    d = {i: dev(v) for i, v in c.items()}
    base = pbg.lora_add(**d)
    out = pbg.lora_add(**{**d, "x": dev(x)})
    keep = torch.from_numpy(~odd).to("cuda:0")
    assert torch.equal(out[keep], base[keep])
    with np.errstate(invalid="ignore"):
        ref, bound = oracle.lora_add(**{**c, "x": x}), lora_bound({**c, "x": x})
    out, ok = host(out).astype(np.float64), np.isfinite(ref)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    assert_within(out[ok], ref[ok], bound[ok], "odd rows")
