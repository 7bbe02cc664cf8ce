"""The linear layer with one adapter per token, forward and backward, against the formulas in fp64.

Tolerances count roundings.  The products of two 16-bit numbers are exact in fp32; a sum of n of them
on the tensor cores takes n / 16 accumulation steps, each off by at most 2^-23 of the running sum of
magnitudes S.  The fp32 factor U (or dU) enters the products as two 16-bit halves, off by 2^-17 of
it in bf16, and by 2^-22 of it plus half of the smallest subnormal, 2^-25, in fp16.  Outputs of a
16-bit type add half a step.
"""
import ctypes
import math

import pytest
import torch

import bit_nf4_quantized_23_b200 as q4
from bit_nf4_quantized_23_b200 import _lib

E = {v: k for k, v in _lib.STATUS_NAMES.items()}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_nf4_quantized_23_b200.build import build
    build()


# ---------------------------------------------------------------------------- host

FAKE = 0x7f0000000000      # never dereferenced: every call below fails validation first


def _w(N=48, K=128, dt=0):
    return _lib.NF4WeightC(0x10000, 0x20000, 0x30000, 0x40000, N, K, 64, 256, 0, dt)


def test_refusals_on_the_host():
    L = _lib.lib()
    before = L.qlora_launch_count()
    w, big = _w(), 1 << 40

    def fwd(w=w, X=FAKE, M=20, A=FAKE, B=FAKE, n=3, idx=FAKE, r=8, s=FAKE, Y=FAKE, dt=0, U=None, ws=FAKE, wb=big):
        return L.qlora_linear_fwd_adapters(ctypes.byref(w), X, M, A, B, n, idx, r, s, Y, dt, U, ws, wb, None)

    def bwd(w=w, X=FAKE, M=20, A=FAKE, B=FAKE, n=3, idx=FAKE, r=8, s=FAKE, U=None, dt=0, ws=FAKE, wb=big, dY=FAKE,
            dX=FAKE, dA=FAKE, dB=FAKE):
        return L.qlora_linear_bwd_adapters(ctypes.byref(w), X, dY, M, A, B, n, idx, r, s, U, dX, dt, dA, dB, ws, wb, None)

    for f in (fwd, bwd):
        for name in ("X", "A", "B", "idx", "s"):
            assert f(**{name: None}) == E["QLORA_ERR_INVALID_ARG"], name
        for name in ("X", "A", "B", "U", "ws"):
            assert f(**{name: FAKE + 8}) == E["QLORA_ERR_ALIGN"], name
        assert f(idx=FAKE + 2) == f(s=FAKE + 1) == E["QLORA_ERR_ALIGN"]
        assert f(r=0) == f(r=257) == f(n=0) == f(n=65536) == f(dt=2) == f(dt=9) == E["QLORA_ERR_INVALID_ARG"]
        assert f(M=0) == f(M=1 << 31) == f(w=_w(K=96)) == f(w=_w(N=1 << 20), n=4096) == E["QLORA_ERR_SHAPE"]
        assert f(ws=None) == f(wb=100) == E["QLORA_ERR_WORKSPACE"]
    assert fwd(Y=None) == bwd(dY=None) == bwd(dA=None) == bwd(dB=None) == E["QLORA_ERR_INVALID_ARG"]
    assert bwd(dX=FAKE + 8) == E["QLORA_ERR_ALIGN"]
    n = ctypes.c_size_t()
    assert L.qlora_adapters_workspace_size(20, 48, 128, 8, 3, None) == E["QLORA_ERR_INVALID_ARG"]
    assert L.qlora_adapters_workspace_size(20, 48, 128, 8, 3, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(wb=n.value - 1) == bwd(wb=n.value - 1) == E["QLORA_ERR_WORKSPACE"]
    assert L.qlora_launch_count() == before


def test_binding_refuses_wrong_tensors():
    w = q4.NF4Weight.empty(48, 128, device="cpu")
    X, A, B = (torch.zeros(s, dtype=BF16) for s in ((5, 128), (2, 8, 128), (2, 48, 8)))
    with pytest.raises(ValueError):                              # not on a CUDA device
        q4.qlora_linear_fwd_adapters(w, X, A, B, torch.zeros(5, dtype=torch.int32), torch.ones(2))


# ---------------------------------------------------------------------------- GPU


class Case:
    """Inputs of one layer; `rows` lays out the adapters: "runs" (contiguous requests), "mixed" (any
    order), "one" (a single adapter), "none"."""

    def __init__(self, M, N, K, r, n, rows="runs", dt=BF16, seed=0, dq=True):
        g = torch.Generator().manual_seed(1000 * seed + M + N + K + r)

        def normal(shape, std):
            return (torch.randn(shape, generator=g) * std).to(dt).cuda()

        self.w = q4.qlora_quantize_nf4_dq((torch.randn(N, K, generator=g) * 0.03).to(BF16).cuda(), double_quant=dq,
                                          compute_dtype=dt)
        self.X, self.dY = normal((M, K), 1.0), normal((M, N), 0.5)
        self.A, self.B = normal((n, r, K), K ** -0.5), normal((n, N, r), 0.2)
        self.scales = (torch.rand(n, generator=g) + 0.5).cuda()
        if rows == "runs":
            cuts = torch.randint(0, M + 1, (2 * n,), generator=g).sort().values.tolist()
            idx = torch.full((M,), -1, dtype=torch.int32)
            for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
                idx[a:b] = int(torch.randint(-1, n, (1,), generator=g))
            idx[0] = n - 1
        elif rows == "mixed":
            idx = torch.randint(-1, n, (M,), generator=g).int()
        else:
            idx = torch.full((M,), 0 if rows == "one" else -1, dtype=torch.int32)
        self.idx, self.dt, self.n, self.r = idx.cuda(), dt, n, r
        self.Wd = q4.qlora_dequantize(self.w).double().cpu()

    def reference(self, U=None):
        """Exact values of the formulas and, for each, the tolerance of an fp32 result."""
        X, dY, A, B = (v.double().cpu() for v in (self.X, self.dY, self.A, self.B))
        s, idx, W, r = self.scales.double().cpu(), self.idx.cpu(), self.Wd, self.r
        M, K, N = X.shape[0], X.shape[1], dY.shape[1]
        eh, ah = (2.0 ** -17, 0.0) if self.dt == BF16 else (2.0 ** -22, 2.0 ** -25)   # the two halves of U and dU
        eg, ag = 2.0 ** -24, (0.0 if self.dt == BF16 else 2.0 ** -47)                 # the three parts
        step = lambda n: (n / 16 + 16) * 2.0 ** -23
        out = {"Y": X @ W.t(), "U": torch.zeros(M, r).double(), "dX": dY @ W, "dA": torch.zeros(self.n, r, K).double(),
               "dB": torch.zeros(self.n, N, r).double()}
        tol = {"Y": step(K + 2 * r + 64) * (X.abs() @ W.abs().t()), "U": torch.zeros(M, r).double(),
               "dX": step(N + 2 * r + 64) * (dY.abs() @ W.abs()), "dA": torch.zeros(self.n, r, K).double(),
               "dB": torch.zeros(self.n, N, r).double()}
        for a in range(self.n):
            m = (idx == a).nonzero()[:, 0]
            if not len(m):
                continue
            Ua = X[m] @ A[a].t()
            tU = step(K) * (X[m].abs() @ A[a].abs().t())
            dU = s[a] * (dY[m] @ B[a])
            rdU = s[a] * step(N) * (dY[m].abs() @ B[a].abs())
            tdU, tsU = rdU + eh * dU.abs() + ah, s[a] * tU + eh * (s[a] * Ua).abs() + ah
            gdU, gsU = rdU + eg * dU.abs() + ag, s[a] * tU + eg * (s[a] * Ua).abs() + ag
            out["U"][m], tol["U"][m] = Ua, tU
            out["Y"][m] += s[a] * Ua @ B[a].t()
            tol["Y"][m] += tsU @ B[a].abs().t() + step(K + 2 * r + 64) * (s[a] * Ua).abs() @ B[a].abs().t()
            out["dX"][m] += dU @ A[a]
            tol["dX"][m] += tdU @ A[a].abs() + step(N + 2 * r + 64) * dU.abs() @ A[a].abs()
            out["dA"][a] = dU.t() @ X[m]
            tol["dA"][a] = gdU.t() @ X[m].abs() + step(2 * M) * (dU.abs().t() @ X[m].abs())
            out["dB"][a] = s[a] * dY[m].t() @ Ua
            tol["dB"][a] = dY[m].abs().t() @ gsU + step(2 * M) * (dY[m].abs().t() @ (s[a] * Ua).abs())
        return out, tol

    def fwd(self, **k):
        return q4.qlora_linear_fwd_adapters(self.w, self.X, self.A, self.B, self.idx, self.scales, **k)

    def bwd(self, **k):
        return q4.qlora_linear_bwd_adapters(self.w, self.X, self.dY, self.A, self.B, self.idx, self.scales, **k)


def close(name, got, ref, tol):
    assert tuple(got.shape) == tuple(ref.shape), name
    half = torch.finfo(got.dtype).eps / 2
    room = tol * (1 + half) + half * ref.abs() + (2.0 ** -25 if got.dtype == F16 else 1e-38)
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all(), name
    assert torch.all(err <= room), (name, float((err / room).max()), (err > room).nonzero()[:4].tolist())


def check(c, out_dtype=None):
    ref, tol = c.reference()
    Y, U = c.fwd(y_dtype=out_dtype)
    close("U", U, ref["U"], tol["U"])
    close("Y", Y, ref["Y"], tol["Y"])
    for saved in (U, None):
        dX, dA, dB = c.bwd(U_saved=saved, dx_dtype=out_dtype)
        close("dA", dA, ref["dA"], tol["dA"])
        close("dB", dB, ref["dB"], tol["dB"])
        close("dX", dX, ref["dX"], tol["dX"])
    assert q4.qlora_read_device_errors(clear=True) == 0


SHAPES = [(1, 1, 64, 1, 1), (1, 64, 64, 8, 3), (16, 130, 128, 3, 4), (17, 130, 128, 3, 4), (40, 256, 320, 16, 40),
          (100, 1000, 1024, 8, 3), (128, 72, 256, 33, 5), (129, 72, 256, 32, 5), (256, 264, 192, 16, 30),
          (257, 264, 192, 64, 6), (300, 520, 1088, 96, 5), (513, 523, 640, 24, 7), (700, 96, 320, 200, 2),
          (1100, 280, 128, 256, 3), (1536, 512, 512, 12, 64)]


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors_on_the_gpu():
    c = Case(20, 136, 128, 8, 3, "mixed")
    for name, bad, error in (("X", c.X[:, :64], ValueError), ("X", c.X.half(), TypeError), ("A", c.A[0], ValueError),
                             ("A", c.A[:, :4], ValueError), ("B", c.B[:2], ValueError), ("idx", c.idx.long(), TypeError),
                             ("idx", c.idx[:5], ValueError), ("scales", c.scales.cpu(), ValueError),
                             ("scales", c.scales.half(), TypeError), ("dY", c.dY.t(), ValueError)):
        good = getattr(c, name)
        setattr(c, name, bad)
        with pytest.raises(error):
            c.bwd()
        if name != "dY":
            with pytest.raises(error):
                c.fwd()
        setattr(c, name, good)
    with pytest.raises(ValueError):
        c.fwd(workspace=torch.empty(16, dtype=torch.uint8))
    with pytest.raises(q4.QloraError):
        c.fwd(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        c.fwd(y_dtype=torch.float64)
    with pytest.raises(q4.QloraError):
        c.fwd(y_dtype=F16)                                       # not the weight's 16-bit type


@pytest.mark.gpu
@pytest.mark.parametrize("rows", ["runs", "mixed"])
@pytest.mark.parametrize("M,N,K,r,n", SHAPES)
def test_forward_and_backward(M, N, K, r, n, rows):
    check(Case(M, N, K, r, n, rows))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n", [(2, 5, 64, 3, 2), (31, 4200, 192, 16, 9), (33, 1000, 2112, 48, 8), (64, 131, 1024, 7, 64),
                                       (65, 2000, 320, 200, 3), (96, 40, 4096, 130, 40), (113, 20000, 128, 64, 2),
                                       (128, 700, 704, 256, 128)])
def test_few_tokens(M, N, K, r, n):
    """Up to 128 tokens take kernels of their own: odd numbers of 64-wide blocks, ranks that are no power
    of two, an adapter per token, one tile for all CTAs and many tiles each."""
    c = Case(M, N, K, r, n, "mixed", seed=4)
    ref, tol = c.reference()
    for out in (F32, BF16):
        Y, U = c.fwd(y_dtype=out)
        close("U", U, ref["U"], tol["U"])
        close("Y", Y, ref["Y"], tol["Y"])
    Y2, none = c.fwd(save_U=False)
    assert none is None and torch.equal(Y, Y2)
    assert q4.qlora_read_device_errors(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n", [(150, 260, 4096, 8, 3), (70, 4163, 192, 20, 5), (400, 2112, 2112, 96, 4), (530, 136, 3008, 150, 2)])
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (F16, F32)])
def test_few_tiles_and_a_long_reduction(M, N, K, r, n, dt, out):
    """Products whose reduction is split over idle SMs and summed afterwards, odd output sizes among them."""
    check(Case(M, N, K, r, n, "mixed", dt=dt), out)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n", [(129, 4100, 2048, 16, 5), (255, 1500, 1088, 40, 6), (640, 300, 2176, 20, 9), (768, 1050, 192, 64, 4),
                                       (769, 200, 1088, 33, 5), (1280, 72, 64, 100, 3)])
@pytest.mark.parametrize("rows", ["runs", "mixed"])
def test_tiles_that_end_at_or_beside_half_of_their_tokens(M, N, K, r, n, rows):
    """Tiles of 512 tokens of which the last has at most 256, or a few more, whole and split reductions."""
    check(Case(M, N, K, r, n, rows, seed=6))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n,dt", [(112, 28672, 8192, 64, 6, F16), (48, 8192, 8192, 16, 32, BF16), (4, 11008, 4096, 16, 4, BF16),
                                          (700, 8192, 4096, 32, 9, BF16), (200, 4096, 11008, 64, 3, F16)])
def test_full_size_layers_repeat_bit_for_bit(M, N, K, r, n, dt):
    """Long runs of units through every ring, several times: any order of arrival that reaches a result
    shows as a difference, and one run is compared with the formula in fp64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(M)
    rnd = lambda *shape, std=1.0, to=dt: (torch.randn(*shape, generator=g, device="cuda") * std).to(to)
    w = q4.qlora_quantize_nf4_dq(rnd(N, K, std=0.02, to=BF16), compute_dtype=dt, double_quant=M % 8 != 0)
    X, dY, A, B = rnd(M, K), rnd(M, N, std=0.1), rnd(n, r, K, std=K ** -0.5), rnd(n, N, r, std=0.05)
    idx = torch.randint(-1, n, (M,), generator=g, device="cuda").int().sort().values
    scales = torch.rand(n, generator=g, device="cuda") + 0.5
    runs = []
    for i in range(5):
        Y, U = q4.qlora_linear_fwd_adapters(w, X, A, B, idx, scales)
        runs.append((Y, U) + q4.qlora_linear_bwd_adapters(w, X, dY, A, B, idx, scales, U_saved=U))
    for later in runs[1:]:
        for a, b in zip(runs[0], later):
            assert torch.equal(a, b)
    W = q4.qlora_dequantize(w).double()
    Yr, dXr = X.double() @ W.t(), dY.double() @ W
    for a in range(n):
        m = (idx == a).nonzero()[:, 0]
        Yr[m] += float(scales[a]) * (X[m].double() @ A[a].double().t()) @ B[a].double().t()
        dXr[m] += float(scales[a]) * (dY[m].double() @ B[a].double()) @ A[a].double()
    # sums of K or N products, each accumulation step off by 2^-23 of the sum of magnitudes, which for these
    # inputs is below sqrt(count) times the result's own scale; half a step of the type on top
    for name, got, ref, count in (("Y", runs[0][0], Yr, K), ("dX", runs[0][2], dXr, N)):
        scale = float(ref.std())
        off = (got.double() - ref).abs()
        room = torch.finfo(dt).eps / 2 * ref.abs() + (count / 16 + 16) * 2.0 ** -23 * count ** 0.5 * scale + 2.0 ** -15 * scale
        assert torch.all(off <= room), (name, float((off / room).max()))
    assert q4.qlora_read_device_errors(clear=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n,rows", [(600, 40, 64, 2, 9000, "mixed"), (4500, 72, 128, 8, 3, "runs"),
                                            (2100, 136, 64, 16, 700, "mixed"), (4097, 64, 64, 8, 2, "mixed")])
def test_many_adapters_and_many_tokens(M, N, K, r, n, rows):
    check(Case(M, N, K, r, n, rows))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", ["one", "none"])
@pytest.mark.parametrize("M,N,K,r,n", [(5, 130, 128, 8, 2), (90, 200, 256, 16, 3), (600, 264, 192, 40, 2)])
def test_a_single_adapter_and_none_at_all(M, N, K, r, n, rows):
    check(Case(M, N, K, r, n, rows))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,out,dq", [(F16, F16, True), (F16, F32, False), (BF16, F32, True), (BF16, BF16, False)])
@pytest.mark.parametrize("M,N,K,r,n,rows", [(9, 130, 128, 8, 4, "mixed"), (77, 301, 320, 20, 9, "mixed"),
                                            (200, 264, 384, 64, 3, "runs"), (520, 136, 256, 130, 4, "runs")])
def test_types(M, N, K, r, n, rows, dt, out, dq):
    check(Case(M, N, K, r, n, rows, dt=dt, dq=dq), out)


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 48, 100, 160])
def test_small_fp16_gradients_keep_their_digits(r):
    """dU of about 1e-5, under fp16's normal numbers, as early in training when B is near zero.  Two parts
    of fp16 alone would be off by 2^-25 / 1e-5, three thousandths; 2^-18 is far above what an fp32 sum of 200
    terms loses."""
    c = Case(200, 136, 192, r, 3, "runs", dt=F16)
    c.dY.mul_(1e-3)
    c.B.mul_(1e-2)
    ref, tol = c.reference()
    _, dA, dB = c.bwd()
    close("dA", dA, ref["dA"], tol["dA"])
    close("dB", dB, ref["dB"], tol["dB"])
    rel = lambda x, y: float((x.double().cpu() - y).norm() / y.norm())
    assert rel(dA, ref["dA"]) <= 2.0 ** -18 and rel(dB, ref["dB"]) <= 2.0 ** -18


@pytest.mark.gpu
@pytest.mark.parametrize("M", [13, 100, 700])
def test_inf_and_nan_stay_in_their_own_request(M):
    c = Case(M, 264, 256, 16, 4, "mixed", seed=3)
    c.idx[:4] = torch.tensor([0, 1, -1, 2], dtype=torch.int32, device="cuda")
    Y, U = c.fwd()
    dX, dA, dB = c.bwd(U_saved=U)
    bad = (c.idx == 1).nonzero()[:, 0]
    c.X[bad], c.dY[bad] = float("nan"), float("inf")
    c.A[1], c.B[1] = float("inf"), float("nan")
    Y2, U2 = c.fwd()
    dX2, dA2, dB2 = c.bwd(U_saved=U2)
    good = (c.idx != 1).nonzero()[:, 0]
    for a, b in ((Y, Y2), (U, U2), (dX, dX2)):
        assert torch.equal(a[good], b[good])
        assert not torch.isfinite(b[bad]).any()
    keep = [0, 2, 3]
    assert torch.equal(dA[keep], dA2[keep]) and torch.equal(dB[keep], dB2[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [10, 300])
def test_an_index_out_of_range_is_flagged_and_uses_the_base(M):
    c = Case(M, 136, 128, 8, 3, "mixed")
    c.idx[:3] = -1
    Y, U = c.fwd()
    g = c.bwd(U_saved=U)
    q4.qlora_read_device_errors(clear=True)
    c.idx[0], c.idx[1], c.idx[2] = 3, 2 ** 31 - 1, -(2 ** 31)
    Y2, U2 = c.fwd()
    assert q4.qlora_read_device_errors(clear=True) == 4
    g2 = c.bwd(U_saved=U2)
    assert q4.qlora_read_device_errors(clear=True) == 4
    assert torch.equal(Y, Y2) and torch.equal(U, U2)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


@pytest.mark.gpu
def test_every_output_is_overwritten_and_the_workspace_may_hold_anything():
    c = Case(330, 264, 192, 16, 5, "runs", seed=1)
    c.idx[c.idx == 2] = 1                                        # adapter 2 has no token
    n = q4.qlora_adapters_workspace_size(330, 264, 192, 16, 5)
    outs = []
    for fill in (0, 255):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        nan = lambda *s, dt=F32: torch.full(s, float("nan"), dtype=dt, device="cuda")
        Y, U = c.fwd(workspace=ws[:n], out=nan(330, 264, dt=BF16), U_out=nan(330, 16))
        g = c.bwd(U_saved=U, workspace=ws[:n], dX=nan(330, 192, dt=BF16), dA=nan(5, 16, 192), dB=nan(5, 264, 16))
        assert torch.all(ws[n:] == fill)
        outs.append((Y, U) + g)
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert torch.all(outs[0][3][2] == 0) and torch.all(outs[0][4][2] == 0)


@pytest.mark.gpu
def test_zero_padded_ranks_equal_the_smaller_adapter():
    small = Case(140, 136, 128, 8, 2, "runs")
    wide = Case(140, 136, 128, 40, 2, "runs")
    for name in ("w", "X", "dY", "idx", "scales", "Wd"):
        setattr(wide, name, getattr(small, name))
    wide.A.zero_(), wide.B.zero_()
    wide.A[:, :8], wide.B[:, :, :8] = small.A, small.B
    ref, tol = small.reference()
    Y, U = wide.fwd()
    dX, dA, dB = wide.bwd(U_saved=U)
    close("Y", Y, ref["Y"], tol["Y"])
    close("dX", dX, ref["dX"], tol["dX"])
    close("dA", dA[:, :8], ref["dA"], tol["dA"])
    close("dB", dB[:, :, :8], ref["dB"], tol["dB"])
    assert torch.all(U[:, 8:] == 0) and torch.all(dA[:, 8:] == 0) and torch.all(dB[:, :, 8:] == 0)


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of <dY, Y> in fp64: Y is linear in A and in B, so they are exact but for
    the rounding of the quotient."""
    c = Case(60, 72, 128, 8, 3, "mixed", seed=2)
    _, tol = c.reference()
    _, dA, dB = c.bwd()
    dY, h = c.dY.double().cpu(), 2.0 ** -4
    for name, grad, at in (("A", dA, (1, 3, 77)), ("A", dA, (0, 7, 5)), ("B", dB, (2, 71, 0)), ("B", dB, (1, 0, 6))):
        t = getattr(c, name)
        val = []
        for sign in (1, -1):
            moved = t.double().cpu()
            moved[at] += sign * h
            setattr(c, name, moved)
            val.append(float((c.reference()[0]["Y"] * dY).sum()))
        setattr(c, name, t)
        num = (val[0] - val[1]) / (2 * h)
        assert abs(num - float(grad[at])) <= float(tol["d" + name][at]) + 1e-9 * max(map(abs, val))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [11, 64, 400])
def test_capture_and_replay_on_a_side_stream_with_new_inputs(M):
    a, b = Case(M, 264, 256, 16, 6, "runs", seed=5), Case(M, 264, 256, 16, 6, "mixed", seed=6)
    X, dY, idx = a.X.clone(), a.dY.clone(), a.idx.clone()
    ws = torch.empty(q4.qlora_adapters_workspace_size(M, 264, 256, 16, 6), dtype=torch.uint8, device="cuda")
    out = dict(Y=torch.empty(M, 264, dtype=BF16, device="cuda"), U=torch.empty(M, 16, device="cuda"),
               dX=torch.empty(M, 256, dtype=BF16, device="cuda"), dA=torch.empty(6, 16, 256, device="cuda"),
               dB=torch.empty(6, 264, 16, device="cuda"))

    def step():
        q4.qlora_linear_fwd_adapters(a.w, X, a.A, a.B, idx, a.scales, out=out["Y"], U_out=out["U"], workspace=ws)
        q4.qlora_linear_bwd_adapters(a.w, X, dY, a.A, a.B, idx, a.scales, U_saved=out["U"], dX=out["dX"],
                                     dA=out["dA"], dB=out["dB"], workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for src in (b, a):
        X.copy_(src.X), dY.copy_(src.dY), idx.copy_(src.idx)
        g.replay()
        torch.cuda.synchronize()
        Y, U = q4.qlora_linear_fwd_adapters(a.w, src.X, a.A, a.B, src.idx, a.scales)
        want = (Y, U) + q4.qlora_linear_bwd_adapters(a.w, src.X, src.dY, a.A, a.B, src.idx, a.scales, U_saved=U)
        for name, v in zip(out, want):
            assert torch.equal(out[name], v), name


@pytest.mark.gpu
def test_two_calls_at_once_and_arguments_that_start_anywhere():
    """Two streams with workspaces of their own, many calls in flight on each, against the same calls one
    after the other; adapter_idx and scales start 4 bytes into their tensors."""
    cases = [Case(90, 2048, 1024, 16, 7, "mixed", seed=11), Case(600, 1024, 2048, 32, 5, "runs", seed=12)]
    for c in cases:
        c.idx = torch.cat([c.idx[:1], c.idx])[1:]
        c.scales = torch.cat([c.scales[:1], c.scales])[1:]
        assert c.idx.data_ptr() % 16 == 4 and c.scales.data_ptr() % 16 == 4
    want = []
    for c in cases:
        Y, U = c.fwd()
        want.append((Y, U) + c.bwd(U_saved=U))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for i in range(6):
        for k, c in enumerate(cases):
            with torch.cuda.stream(streams[k]):
                Y, U = c.fwd()
                got[k].append((Y, U) + c.bwd(U_saved=U, stream=streams[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            for a, b in zip(want[k], run):
                assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n", [(5, 264, 192, 16, 3), (60, 2048, 1024, 24, 5), (200, 512, 2048, 8, 4), (600, 256, 320, 32, 6)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_buffers_aligned_to_sixteen_bytes_only(M, N, K, r, n, out):
    """Every buffer may start at any multiple of 16 bytes; the results are those of other starts, bit for bit."""
    def shifted(shape, dtype):
        size = math.prod(shape) * dtype.itemsize
        raw = torch.full((size + 48,), 0xFF, dtype=torch.uint8, device="cuda")
        at = 16 if raw.data_ptr() % 32 == 0 else 0
        return raw[at:at + size].view(dtype).view(shape)

    c = Case(M, N, K, r, n, "mixed", seed=15)
    Y, U = c.fwd(y_dtype=out)
    dX, dA, dB = c.bwd(U_saved=U, dx_dtype=out)
    ws = shifted((q4.qlora_adapters_workspace_size(M, N, K, r, n),), torch.uint8)
    Y2, U2 = c.fwd(y_dtype=out, out=shifted((M, N), out), U_out=shifted((M, r), F32), workspace=ws)
    for name in ("X", "dY", "A", "B"):
        v = getattr(c, name)
        setattr(c, name, shifted(tuple(v.shape), v.dtype).copy_(v))
    Y3, U3 = c.fwd(y_dtype=out, workspace=ws)
    got = c.bwd(U_saved=U2, dx_dtype=out, dX=shifted((M, K), out), dA=shifted((n, r, K), F32), dB=shifted((n, N, r), F32),
                workspace=ws)
    assert all(t.data_ptr() % 32 == 16 for t in (ws, Y2, U2, c.X, c.dY, c.A, c.B) + got)
    for a, b in zip((Y, U, Y, U, dX, dA, dB), (Y2, U2, Y3, U3) + got):
        assert torch.equal(a, b)
    assert q4.qlora_read_device_errors(clear=True) == 0


@pytest.mark.gpu
def test_need_dX_false_and_a_chain_through_the_distillation_loss():
    """An output projection with the adapters of three jobs, the loss of its logits against a teacher's
    top logits, and the backward through both; the gradients against the same chain in fp64 from the
    kernels' own logits."""
    M, V, K, r, n, k, T = 150, 1000, 256, 16, 3, 12, 2.0
    c = Case(M, V, K, r, n, "runs", seed=8)
    g = torch.Generator().manual_seed(1)
    t_idx = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(M)]).int().cuda()
    t_val = (torch.randn(M, k, generator=g) * 2).cuda()
    t_idx[7] = -1
    logits, U = c.fwd(y_dtype=F32)
    loss, lse = q4.qlora_distill_topk_fwd(logits, t_idx, t_val, T)
    c.dY = q4.qlora_distill_topk_bwd(logits, t_idx, t_val, lse, torch.full((M,), 1.0 / M, device="cuda"), T, d_dtype=BF16)
    ref, tol = c.reference()
    dX, dA, dB = c.bwd(U_saved=U)
    close("dX", dX, ref["dX"], tol["dX"])
    close("dA", dA, ref["dA"], tol["dA"])
    close("dB", dB, ref["dB"], tol["dB"])
    none, dA2, dB2 = c.bwd(U_saved=U, need_dX=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    # the chain's total derivative along a direction in B: differences of the mean loss in fp64
    D = torch.randn(n, V, r, generator=g).double() * 0.05
    X64, A64, B64 = c.X.double().cpu(), c.A.double().cpu(), c.B.double().cpu()
    ids, s = c.idx.cpu(), c.scales.double().cpu()

    def mean_loss(B):
        z = X64 @ c.Wd.t()
        for a in range(n):
            m = (ids == a).nonzero()[:, 0]
            z[m] += s[a] * (X64[m] @ A64[a].t()) @ B[a].t()
        logq = torch.log_softmax(z / T, 1)
        p = torch.softmax(t_val.double().cpu() / T, 1)
        li = T * T * (p * (p.log() - logq.gather(1, t_idx.clamp(min=0).long().cpu()))).sum(1)
        li[7] = 0
        return float(li.mean())

    h = 1e-3
    num = (mean_loss(B64 + h * D) - mean_loss(B64 - h * D)) / (2 * h)
    got = float((dB.double().cpu() * D).sum())
    # dY is rounded to bf16 (half a step each, independent of D's signs in sum at most sum |dB D| 2^-8);
    # the difference quotient's own error is below h^2
    bound = float((c.dY.double().cpu().abs().t() @ U.double().cpu().abs()).mul(D.abs().amax(0) * s.max()).sum()) * 2.0 ** -8
    assert abs(num - got) <= bound + 1e-5, (num, got, bound)


def _with_switch(code, **env):
    """Standard output of `code` in a process of its own, since the switches are read once."""
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    root = os.path.dirname(tests)
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600,
                         env={**os.environ, "PYTHONPATH": os.pathsep.join([root, tests]), **env})
    assert res.returncode == 0, res.stderr[-2000:]
    return res.stdout


def test_the_switch_to_single_cta_kernels_covers_the_adapter_calls():
    """200 tokens through W[8192, 8192] split the reduction over pairs, for which the workspace holds fp32
    partial outputs; with QLORA_PAIR_GEMM=0 there are none (on the host: the size is all that is asked)."""
    code = ("import bit_nf4_quantized_23_b200 as q4; "
            "print(q4.qlora_adapters_workspace_size(200, 8192, 8192, 16, 4), q4.qlora_adapters_workspace_size(2, 64, 64, 16, 4))")
    with_pairs, without = (_with_switch(code, QLORA_PAIR_GEMM=v).split() for v in ("1", "0"))
    assert int(with_pairs[0]) - int(without[0]) >= 2 * 200 * 8192 * 4
    assert with_pairs[1] == without[1]


@pytest.mark.gpu
@pytest.mark.parametrize("env", [dict(QLORA_PAIR_GEMM="0"), dict(QLORA_PAIR_BN="240"), dict(QLORA_PAIR_BN="224")])
def test_results_under_the_switches(env):
    code = """
import torch
from test_adapters import BF16, F16, F32, Case, check
for shape in [(100, 136, 256, 16, 4), (129, 300, 192, 40, 3), (256, 264, 192, 16, 30), (300, 520, 1088, 96, 5),
              (513, 523, 640, 24, 7), (1100, 280, 128, 256, 3)]:
    for rows in ("runs", "mixed"):
        check(Case(*shape, rows))
check(Case(700, 264, 384, 64, 3, "mixed", dt=F16), F32)
print("as the formulas")
"""
    assert "as the formulas" in _with_switch(code, **env)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,n", [(200, 20000, 128, 16, 5), (256, 28672, 64, 40, 3), (100, 136, 20032, 8, 4),
                                       (129, 72, 20032, 33, 3), (256, 200, 22016, 64, 6)])
@pytest.mark.parametrize("rows", ["runs", "mixed"])
def test_wide_outputs_of_up_to_256_tokens(M, N, K, r, n, rows):
    """75 to 148 tiles of 256 columns: one wave of single CTAs, which these products take, or two of pairs."""
    check(Case(M, N, K, r, n, rows, seed=9))


def test_what_is_no_tensor_is_a_type_error(monkeypatch):
    w = q4.NF4Weight.empty(48, 128, device="cpu")
    X, dY, A, B = (torch.zeros(s, dtype=BF16) for s in ((5, 128), (5, 48), (2, 8, 128), (2, 48, 8)))
    idx, scales = torch.zeros(5, dtype=torch.int32), torch.ones(2)
    monkeypatch.setattr(q4, "_device_of", lambda *a: -1)         # lets tensors of the host past the first check
    good = dict(A_all=A, B_all=B, adapter_idx=idx, scales=scales)
    for name in [*good, "workspace"]:
        args = {**good, name: 3}
        with pytest.raises(TypeError, match=name + " must be a torch.Tensor"):
            q4.qlora_linear_fwd_adapters(w, X, **args)
        with pytest.raises(TypeError, match=name + " must be a torch.Tensor"):
            q4.qlora_linear_bwd_adapters(w, X, dY, **args)


@pytest.mark.gpu
def test_fp32_results_lose_no_more_than_their_chains():
    """The tensor cores cut each running fp32 sum toward zero, at most a step of 2^-23 and on average half of it,
    once for every 16 products.  U, dA and dB are joined from sums of 64 such steps; Y and dX in fp32 are one chain
    over the whole reduction when there are tiles enough for the GPU (the largest loss there is)."""
    M, N, K, r = 2048, 11008, 4864, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)
    w = q4.qlora_quantize_nf4_dq(rnd(N, K, std=0.02))
    X, dY, A, B = rnd(M, K), rnd(M, N), rnd(1, r, K, std=K ** -0.5), torch.zeros(1, N, r, dtype=BF16, device="cuda")
    idx, one = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    Y, U = q4.qlora_linear_fwd_adapters(w, X, A, B, idx, one, y_dtype=F32)
    dX, _, dB = q4.qlora_linear_bwd_adapters(w, X, dY, A, B, idx, one, U_saved=U, dx_dtype=F32)
    W, m = q4.qlora_dequantize(w).double(), slice(0, 128)
    for name, got, ref, steps in (("Y", Y[m], X[m].double() @ W.t(), K / 16), ("dX", dX[m], dY[m].double() @ W, N / 16),
                                  ("U", U, X.double() @ A[0].double().t(), 64),
                                  ("dB", dB[0], dY.double().t() @ U.double(), 64)):
        loss = float(((ref - got.double()) * ref.sign()).sum() / ref.abs().sum())
        assert abs(loss) <= steps * 2.0 ** -24, (name, loss)


@pytest.mark.gpu
@pytest.mark.parametrize("r", [8, 100])
def test_what_a_small_fp16_dU_is_worth_in_dX(r):
    """dU of about 1e-5 enters dX as two halves of fp16, together off by at most 2^-25: a few thousandths of such a
    dU, and far below fp16's smallest number in dX itself.  The weight is zero, so that dX is the adapter's term."""
    c = Case(200, 136, 192, r, 3, "runs", dt=F16)
    c.w = q4.qlora_quantize_nf4_dq(torch.zeros(136, 192, dtype=BF16, device="cuda"), compute_dtype=F16)
    c.Wd = q4.qlora_dequantize(c.w).double().cpu()
    assert torch.all(c.Wd == 0)
    c.dY.mul_(1e-3)
    c.B.mul_(1e-2)
    ref, _ = c.reference()
    dX, _, _ = c.bwd(dx_dtype=F32)
    # on top: sums of N and of 2 r products of fp32, at most 2^-23 of their magnitudes a step
    s, idx, mag = c.scales.double().cpu(), c.idx.cpu(), torch.zeros_like(ref["dX"])
    floor = torch.zeros_like(mag)
    for a in range(3):
        m = (idx == a).nonzero()[:, 0]
        A = c.A[a].double().cpu().abs()
        mag[m] = s[a] * (c.dY[m].double().cpu().abs() @ c.B[a].double().cpu().abs()) @ A
        floor[m] = 2.0 ** -25 * A.sum(0)
    assert torch.all((dX.double().cpu() - ref["dX"]).abs() <= floor + 40 * 2.0 ** -23 * mag)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F16])
def test_dB_of_a_long_batch_keeps_fp32_digits(dt):
    """One adapter with 2048 tokens.  32 steps of the tensor cores, each of which loses 2^-26 of the running sum,
    are 5e-7; the three parts of U (2^-24) and four fp32 additions (2^-24 each, either way) stay below 2e-7."""
    c = Case(2048, 520, 512, 16, 1, "one", dt=dt)
    U = (c.X.double() @ c.A[0].double().t()).float()
    _, _, dB = c.bwd(U_saved=U)
    ref = float(c.scales[0]) * c.dY.double().t() @ U.double()
    assert float((dB[0].double() - ref).norm() / ref.norm()) <= 7e-7
