"""The distillation loss from a teacher's top logits and its gradient, against the formulas in fp64.

Tolerances count roundings.  With Y the largest |z / T| log2(e) of a row, the exponent of an element
is off by at most 3 Y 2^-24 (the constant, the reference and the fused multiply-add are each rounded),
an exponential by 2^-22 more, and the sum of V of them by (V / 256 + 32) 2^-24 (each of 256 threads
adds its share, a tree joins them).  E = (4 Y + V / 256 + 64) 2^-24 bounds the sum of these for lse
and for log q; the teacher's side has the same bound with its own exponents.
"""
import math

import pytest
import torch

import bit_nf4_quantized_23_b200 as q4
from bit_nf4_quantized_23_b200 import _lib

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E = {v: k for k, v in _lib.STATUS_NAMES.items()}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_nf4_quantized_23_b200.build import build
    build()


# ---------------------------------------------------------------------------- host

FAKE = 0x7f0000000000      # never dereferenced: every call below fails validation first


def test_refusals_on_the_host():
    L = _lib.lib()
    before = L.qlora_launch_count()

    def fwd(z=FAKE, zt=0, ld=100, M=4, V=100, idx=FAKE, t=FAKE, tt=1, k=8, T=1.0, loss=FAKE, lse=FAKE):
        return L.qlora_distill_topk_fwd(z, zt, ld, M, V, idx, t, tt, k, T, loss, lse, None)

    def bwd(z=FAKE, zt=0, ld=104, M=4, V=100, idx=FAKE, t=FAKE, tt=1, k=8, T=1.0, lse=FAKE, dl=FAKE,
            d=FAKE + (1 << 20), dt=0, ldd=104):
        return L.qlora_distill_topk_bwd(z, zt, ld, M, V, idx, t, tt, k, T, lse, dl, d, dt, ldd, None)

    for f in (fwd, bwd):
        assert f(z=None) == E["QLORA_ERR_INVALID_ARG"]
        assert f(z=FAKE + 1) == f(z=FAKE + 2, zt=1) == f(lse=FAKE + 2) == E["QLORA_ERR_ALIGN"]
        assert f(idx=None) == E["QLORA_ERR_INVALID_ARG"]
        assert f(t=FAKE + 2) == E["QLORA_ERR_ALIGN"]
        assert f(lse=None) == E["QLORA_ERR_INVALID_ARG"]
        assert f(zt=3) == f(tt=-1) == E["QLORA_ERR_INVALID_ARG"]
        assert f(k=0) == f(k=1025) == E["QLORA_ERR_INVALID_ARG"]
        for T in (0.0, -1.0, 1e-4, 1e4, float("nan"), float("inf")):
            assert f(T=T) == E["QLORA_ERR_INVALID_ARG"]
        assert f(M=0) == f(V=0) == f(ld=99) == f(V=1 << 31, ld=1 << 31) == f(ld=1 << 39) == E["QLORA_ERR_SHAPE"]
    assert fwd(loss=None) == E["QLORA_ERR_INVALID_ARG"]
    assert bwd(d=None) == bwd(dt=9) == bwd(dl=None) == E["QLORA_ERR_INVALID_ARG"]
    assert bwd(ldd=99) == E["QLORA_ERR_SHAPE"]
    # overlaps: another stride, another element size, a shifted start, the end of the logits
    for bad in (dict(d=FAKE, ldd=112), dict(d=FAKE, dt=1), dict(d=FAKE + 16), dict(d=FAKE + 816)):
        assert bwd(**bad) == E["QLORA_ERR_INVALID_ARG"]
    assert L.qlora_launch_count() == before


def test_binding_refuses_wrong_tensors():
    z, i, t = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        q4.qlora_distill_topk_fwd(z, i, t)                       # not on a CUDA device
    with pytest.raises(TypeError):
        q4.qlora_distill_topk_fwd([0.0], i, t)


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors_on_the_gpu():
    z, i, t = torch.zeros(2, 8).cuda(), torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.zeros(2, 3).cuda()
    v = torch.zeros(2).cuda()
    for bad, error in (((z[0], i, t), ValueError), ((z.double(), i, t), TypeError), ((z.t(), i, t), ValueError),
                       ((z, i.long(), t), TypeError), ((z, i[:1], t), ValueError), ((z, i, t[:, :2]), ValueError),
                       ((z, i.cpu(), t), ValueError)):
        with pytest.raises(error):
            q4.qlora_distill_topk_fwd(*bad)
    for bad in ((z, i, t, v[:1], v), (z, i, t, v, v[:1])):
        with pytest.raises(ValueError):
            q4.qlora_distill_topk_bwd(*bad)
    with pytest.raises(ValueError):
        q4.qlora_distill_topk_bwd(z, i, t, v, v, dlogits=z[:1])
    with pytest.raises(TypeError):
        q4.qlora_distill_topk_bwd(z, i, t, v, v, d_dtype=torch.bfloat16, dlogits=z)


# ---------------------------------------------------------------------------- GPU


def formulas(z, idx, t, T, dloss):
    """(loss, lse, dz, sum_j p |log p - log q|) in fp64, row by row."""
    z, t = z.double().cpu(), t.double().cpu()
    idx, M, V = idx.cpu(), z.shape[0], z.shape[1]
    loss, lse, dz, mag = torch.zeros(M).double(), torch.zeros(M).double(), torch.zeros(M, V).double(), torch.zeros(M).double()
    for m in range(M):
        y = z[m] / T
        top = y[~y.isnan()].max()
        lse[m] = top + (y - top).exp().sum().log()
        ok = (idx[m] >= 0) & (idx[m] < V) & (t[m] > -math.inf)
        if not ok.any():
            continue
        p = torch.softmax(t[m][ok] / T, 0)
        i = idx[m][ok].long()
        d = torch.where(p > 0, p.log() - (y[i] - lse[m]), torch.zeros(()).double())
        loss[m] = T * T * (torch.where(p > 0, p * d, torch.zeros(()).double())).sum()
        mag[m] = T * T * (p * d).abs().nan_to_num(0.0).sum()
        if dloss[m] != 0:
            dz[m] = (y - lse[m]).exp().index_add(0, i, -p) * T * dloss[m].double().cpu()
    return loss, lse, dz, mag


def unit(z, t, idx, T, V):
    zf, tf = z.double().cpu(), t.double().cpu()
    big = max(float(zf[zf.isfinite()].abs().max()), float(tf[tf.isfinite()].abs().max()))
    return (4 * big / T * math.log2(math.e) + V / 256 + 64) * 2.0 ** -24


def make(M, V, k, dt, tdt, seed, pad=0, std=2.5):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(M, V + pad, generator=g) * std).to(dt)[:, :V].cuda() if pad else \
        (torch.randn(M, V, generator=g) * std).to(dt).cuda()
    if pad:
        z = torch.nn.functional.pad(z, (0, pad), value=float("nan"))[:, :V]
    idx = torch.randint(0, V, (M, k), generator=g).int()
    idx[torch.rand(M, k, generator=g) < 0.2] = -1
    t = (torch.randn(M, k, generator=g) * std).to(tdt)
    dloss = torch.rand(M, generator=g) + 0.5
    return z, idx.cuda(), t.cuda(), dloss.cuda()


def check_case(z, idx, t, T, dloss, out_dtype, dlogits=None):
    M, V = z.shape
    ref_loss, ref_lse, ref_dz, mag = formulas(z, idx, t, T, dloss)
    e = unit(z, t, idx, T, V)
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, T)
    zc = z.double().cpu()
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, T, d_dtype=out_dtype, dlogits=dlogits)
    torch.cuda.synchronize()
    assert torch.all((lse.double().cpu() - ref_lse).abs() <= e * (1 + ref_lse.abs()))
    assert torch.all((loss.double().cpu() - ref_loss).abs() <= 2 * e * (T * T + mag) + 2.0 ** -23 * ref_loss.abs())
    # q and each p are off by their exponents' error; both times dloss T; then the rounding to the type
    p_sum = ((zc / T - ref_lse[:, None]).exp() * T * dloss.double().cpu()[:, None] - ref_dz).abs()
    q = (zc / T - ref_lse[:, None]).exp() * T * dloss.double().cpu()[:, None]
    half = torch.finfo(out_dtype).eps / 2
    # below the smallest normal number the step is constant: half of the smallest subnormal
    tiny = torch.finfo(out_dtype).tiny * half + (1e-37 if out_dtype != torch.float16 else 0.0)
    tol = 4 * e * (q + p_sum) + half * ref_dz.abs() + 2 * tiny
    err = (dz.double().cpu() - ref_dz).abs()
    assert dz.dtype == out_dtype
    assert torch.all(err <= tol), float((err / tol).max())
    return loss, lse, dz


@pytest.mark.gpu
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"),
                                    ("fp32", "fp16"), ("bf16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("M,V,k,T", [(1, 1, 1, 1.0), (3, 7, 2, 2.0), (5, 1000, 17, 1.0), (2, 33001, 64, 0.7),
                                     (300, 4099, 33, 4.0)])
def test_loss_and_gradient(dt, out, M, V, k, T):
    z, idx, t, dloss = make(M, V, k, DT[dt], torch.float32, seed=M + V + k)
    check_case(z, idx, t, T, dloss, DT[out])
    assert q4.qlora_read_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tdt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("k", [1, 256, 257, 1024])
def test_teacher_types_and_entry_counts(tdt, k):
    z, idx, t, dloss = make(4, 5000, k, torch.bfloat16, DT[tdt], seed=k)
    check_case(z, idx, t, 1.5, dloss, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("pad,dpad", [(3, 3), (8, 0), (5, 0), (0, 7), (1, 9)])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
def test_row_strides_and_columns_behind_the_row(pad, dpad, dt, out):
    """Rows of a padded head: NaN behind the vocabulary is never read, and the padding of the gradient
    keeps its values (equal strides, strides that agree modulo eight, and strides that do not)."""
    M, V = 5, 1001
    z, idx, t, dloss = make(M, V, 9, DT[dt], torch.float32, seed=11 + pad, pad=pad)
    buf = torch.full((M, V + dpad), 7.0, dtype=DT[out], device="cuda")
    check_case(z, idx, t, 1.0, dloss, DT[out], dlogits=buf[:, :V])
    assert torch.all(buf[:, V:] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("z0,d0", [(0, 0), (1, 1), (3, 0), (2, 6), (5, 1)])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32"), ("bf16", "fp32")])
def test_rows_that_start_anywhere(z0, d0, dt, out):
    """A chunk of rows of a larger tensor with an odd row length starts at any element."""
    M, V, k = 4, 1003, 7
    z, idx, t, dloss = make(M, V, k, DT[dt], torch.float32, seed=z0 + 8 * d0)
    zb = torch.full((M * V + 8,), float("nan"), dtype=DT[dt], device="cuda")
    db = torch.full((M * V + 8,), 7.0, dtype=DT[out], device="cuda")
    zv, dv = (b[o:o + M * V].view(M, V) for b, o in ((zb, z0), (db, d0)))
    zv.copy_(z)
    idx2, t2 = (torch.cat([v.flatten()[:1], v.flatten()])[1:].view(M, k) for v in (idx, t))   # 4 bytes in
    check_case(zv, idx2, t2, 1.0, dloss, DT[out], dlogits=dv)
    assert torch.all(db[:d0] == 7.0) and torch.all(db[d0 + M * V:] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [9, 1001, 40000])
def test_in_place_gradient_equals_the_separate_one(V):
    z, idx, t, dloss = make(6, V, 8, torch.bfloat16, torch.float32, seed=V)
    idx[0] = idx[0, 0].clamp(min=0)                              # one logit eight times
    _, lse = q4.qlora_distill_topk_fwd(z, idx, t, 2.0)
    apart = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, 2.0)
    q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, 2.0, dlogits=z)
    assert torch.equal(apart.view(torch.int16), z.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [6, 400])
def test_rows_without_entries_masks_and_repeated_indices(M):
    V, k = 20011, 12
    z, idx, t, dloss = make(M, V, k, torch.float32, torch.float32, seed=5)
    idx[0] = -1                                                  # no entry
    idx[1] = 777                                                 # the same index k times
    t[2] = -math.inf                                             # every teacher logit masked
    t[3] = torch.finfo(torch.float32).min                        # the lowest value: an even distribution
    t[4, 1:] = -math.inf                                         # one entry left
    dloss[5] = 0.0
    z[0] = math.nan                                              # never read into a row without entries
    z[2, 100] = math.inf
    z[5, 3] = math.nan
    z[1, :5000] = -math.inf                                      # masked vocabulary
    z[4, 5000:] = torch.finfo(torch.float32).min
    idx[4] = torch.arange(k, dtype=torch.int32, device="cuda")
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, 1.0)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, 1.0)
    for m in (0, 2):
        assert loss[m] == 0 and torch.all(dz[m] == 0)
    assert torch.all(dz[5] == 0)
    rows = [1, 3, 4] + list(range(6, M))
    zr, ir, tr, dr = (v[rows].contiguous() for v in (z, idx, t, dloss))
    zs = zr.clone()
    zs[zs == torch.finfo(torch.float32).min] = -math.inf         # e^lowest is 0 as e^-inf is
    tr64 = tr.clone()
    tr64[tr64 == torch.finfo(torch.float32).min] = 0.0
    ref_loss, ref_lse, ref_dz, mag = formulas(zs, ir, tr64, 1.0, dr)
    e = unit(zs, tr64, ir, 1.0, V)
    got = loss[rows].double().cpu()
    # row 1: all of the teacher's weight on a masked logit, a loss of +inf on both sides
    assert got[0] == math.inf and ref_loss[0] == math.inf
    off = (got - ref_loss)[1:].abs()
    assert torch.all(off <= (2 * e * (1 + mag) + 2.0 ** -23 * ref_loss.abs())[1:])
    q = (zs.double().cpu() - ref_lse[:, None]).exp() * dr.double().cpu()[:, None]
    tol = 4 * e * (q + (q - ref_dz).abs()) + 2.0 ** -24 * ref_dz.abs() + 1e-37
    assert torch.all((dz[rows].double().cpu() - ref_dz).abs() <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0.5, 1.0, 30.0])
@pytest.mark.parametrize("M,V", [(5, 9), (5, 30011), (700, 515)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_whose_own_logits_are_all_masked(M, V, T, dt):
    """Such a row has loss 0, gradient 0 and lse -inf; rows beside it, and a row with one logit left, do not."""
    z, idx, t, dloss = make(M, V, 4, dt, torch.float32, seed=3)
    idx[:, 0] = 1
    plain = check_case(z, idx, t, T, dloss, dt)
    z = z.clone()
    z[0] = -math.inf
    z[1] = torch.finfo(dt).min
    z[2, ::2], z[2, 1::2] = -math.inf, torch.finfo(dt).min
    z[3] = torch.finfo(dt).min
    z[3, 1], idx[3, 1:] = 2.5, -1                                # the teacher's one choice is the one logit left
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, T)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, T)
    assert torch.all(lse[:3] == -math.inf) and torch.all(loss[:3] == 0) and torch.all(dz[:3] == 0)
    # q = p = 1: lse is 2.5 / T to four roundings of a value below 8 / T, and all else follows from it
    e = 2.0 ** -22 * 8 / T
    assert abs(float(lse[3]) - 2.5 / T) <= e and abs(float(loss[3])) <= 2 * T * T * e
    assert torch.all(dz[3].float().abs() <= 2 * T * e * dloss[3])
    for new, old in zip((loss, lse, dz), plain):
        assert torch.equal(new[4:], old[4:])


@pytest.mark.gpu
def test_a_teacher_index_behind_the_vocabulary_is_flagged_and_skipped():
    z, idx, t, dloss = make(3, 500, 4, torch.bfloat16, torch.float32, seed=9)
    q4.qlora_read_device_errors(clear=True)
    idx[1, 2] = 500
    check_case(z, idx, t, 1.0, dloss, torch.float32)
    assert q4.qlora_read_device_errors(clear=True) == 4


@pytest.mark.gpu
def test_gradient_against_differences():
    """(loss(z + h e) - loss(z - h e)) / 2h in fp64 of the formula agrees with the kernel's gradient."""
    z, idx, t, _ = make(2, 50, 6, torch.float32, torch.float32, seed=3)
    one = torch.ones(2, device="cuda")
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, 2.0)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, one, 2.0).double().cpu()
    h = 1e-4
    for v in (0, 17, int(idx[0][idx[0] >= 0][0]), 49):
        up, down = z.double().cpu().clone(), z.double().cpu().clone()
        up[:, v] += h
        down[:, v] -= h
        num = (formulas(up, idx, t, 2.0, one)[0] - formulas(down, idx, t, 2.0, one)[0]) / (2 * h)
        # truncation h^2/6 of a third derivative below T^2 / T^3, cancellation 2^-52 |loss| / h, the kernel's own E
        assert torch.all((num - dz[:, v]).abs() <= h * h + 1e-11 + 8 * unit(z, t, idx, 2.0, 50))


@pytest.mark.gpu
def test_capture_and_replay_on_a_side_stream_with_new_inputs():
    s = torch.cuda.Stream()
    a = make(7, 9001, 16, torch.bfloat16, torch.float32, seed=1)
    b = make(7, 9001, 16, torch.bfloat16, torch.float32, seed=2)
    z, idx, t, dloss = (v.clone() for v in a)
    loss, lse = torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    dz = torch.empty_like(z)

    def step():
        q4.qlora_distill_topk_fwd(z, idx, t, 1.0, loss=loss, lse=lse)
        q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, 1.0, dlogits=dz)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for src in (b, a):
        for dst, v in zip((z, idx, t, dloss), src):
            dst.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        want, want_lse = q4.qlora_distill_topk_fwd(*src[:3], 1.0)
        assert torch.equal(loss, want) and torch.equal(lse, want_lse)
        assert torch.equal(dz, q4.qlora_distill_topk_bwd(*src[:3], want_lse, src[3], 1.0))


FINITE_MASKS = [(d, m) for d in (torch.bfloat16, torch.float32) for m in (torch.finfo(d).min, -1e30, -1e10, -1e9)] + \
    [(torch.float16, torch.finfo(torch.float16).min), (torch.float16, -1e4)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [(6, 40011), (300, 5003)])      # a cluster for each row, a CTA for each row
@pytest.mark.parametrize("T", [0.7, 1.0, 1.5, 2.0, 4.0])
@pytest.mark.parametrize("dt,mask", FINITE_MASKS)
def test_finite_masks_count_as_minus_infinity(dt, mask, T, M, V):
    """A masked prefix, masked leading chunks, all but a few scattered logits masked, every second logit
    masked: threads that meet only masks, first or throughout.  exp(mask / T) is 0 in fp64 too, so the
    formula of -inf logits is the reference, with the tolerance of the logits that are left."""
    z, idx, t, dloss = make(M, V, 9, dt, torch.float32, seed=21)
    masked = torch.zeros(M, V, dtype=torch.bool, device="cuda")
    at = torch.arange(V, device="cuda")
    masked[0::6] = at < V // 2
    masked[1::6] = at < V - 20
    masked[2::6] = (at != 17) & (at != V // 3) & (at != V - 2)
    masked[3::6] = at % 2 == 0
    masked[4::6] = at >= 5
    left = [torch.nonzero(~masked[m])[:, 0] for m in range(6)]
    for m in range(M):                                           # the teacher's entries are logits that are left
        idx[m] = torch.where(idx[m] < 0, idx[m], left[m % 6][(idx[m] % len(left[m % 6])).long()].int())
    z = z.masked_fill(masked, mask)
    zs = z.masked_fill(masked, -math.inf)
    ref_loss, ref_lse, ref_dz, mag = formulas(zs, idx, t, T, dloss)
    e = unit(zs, t, idx, T, V)
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, T)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, T, d_dtype=torch.float32)
    assert torch.all((lse.double().cpu() - ref_lse).abs() <= e * (1 + ref_lse.abs()))
    assert torch.all((loss.double().cpu() - ref_loss).abs() <= 2 * e * (T * T + mag) + 2.0 ** -23 * ref_loss.abs())
    q = (zs.double().cpu() / T - ref_lse[:, None]).exp() * T * dloss.double().cpu()[:, None]
    tol = 4 * e * (q + (q - ref_dz).abs()) + 2.0 ** -24 * ref_dz.abs() + 1e-37
    assert torch.all((dz.double().cpu() - ref_dz).abs() <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [9, 30011])
@pytest.mark.parametrize("T", [0.7, 1.0, 1.5, 2.0, 4.0, 30.0])
@pytest.mark.parametrize("dt,mask", [c for c in FINITE_MASKS if c[1] != -1e4])
def test_rows_masked_throughout_by_any_mask(dt, mask, T, V):
    z, idx, t, dloss = make(3, V, 4, dt, torch.float32, seed=4)
    idx[:, 0] = 1
    z[0] = mask
    z[1, ::2], z[1, 1::2] = mask, -math.inf
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, T)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, dloss, T)
    assert torch.all(lse[:2] == -math.inf) and torch.all(loss[:2] == 0) and torch.all(dz[:2] == 0)
    assert torch.isfinite(lse[2]) and torch.isfinite(loss[2]) and torch.any(dz[2] != 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0.7, 1.0, 1.5])
@pytest.mark.parametrize("dt,mask", [c for c in FINITE_MASKS if c[0] != torch.float16])
def test_the_teachers_weight_on_a_masked_logit_costs_its_distance(dt, mask, T):
    """Half of the teacher's weight on a logit at the mask: the loss is T p (z_max - mask) and small terms, finite
    in fp32 for these T although mask / T^2 may not be.  p, its product and the sum are each rounded, and the
    approximation of p is off by 2^-22: 2^-20 in all, of a loss of at least 0.5 T |mask|."""
    V = 3000
    z, _, _, _ = make(2, V, 2, dt, torch.float32, seed=2)
    z[:, 100:] = mask
    idx = torch.tensor([[5, 2000], [2500, 7]], dtype=torch.int32, device="cuda")
    t = torch.zeros(2, 2, device="cuda")
    ref = formulas(z, idx, t, T, torch.ones(2))[0]
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, T)
    assert torch.isfinite(ref.float()).all() and torch.isfinite(lse).all()
    assert torch.all((loss.double().cpu() - ref).abs() <= 2.0 ** -20 * ref)


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [(2, 9), (2, 40011), (300, 5003)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_a_logit_of_plus_infinity_has_the_whole_row(dt, M, V):
    """lse is +inf as logsumexp has it; every other logit has probability 0, so a teacher that wants one of them
    has a loss of +inf and the gradient -p there; inf - inf on the logit itself is NaN.  A NaN in the row wins."""
    z, _, _, _ = make(M, V, 1, dt, torch.float32, seed=6)
    idx = torch.full((M, 1), 2, dtype=torch.int32, device="cuda")
    t, one = torch.zeros(M, 1, device="cuda"), torch.ones(M, device="cuda")
    z[0, V - 4] = math.inf
    z[1, V - 4], z[1, 0] = math.inf, math.nan
    loss, lse = q4.qlora_distill_topk_fwd(z, idx, t, 2.0)
    dz = q4.qlora_distill_topk_bwd(z, idx, t, lse, one, 2.0)
    assert lse[0] == math.inf and loss[0] == math.inf and lse[1].isnan() and loss[1].isnan()
    want = torch.zeros(V, device="cuda")
    want[2], want[V - 4] = -2.0, math.nan
    assert torch.equal(dz[0].float().nan_to_num(9.0), want.nan_to_num(9.0)) and dz[1].isnan().all()
    assert torch.isfinite(lse[2:]).all() and torch.isfinite(dz[2:]).all()


def test_what_is_no_tensor_is_a_type_error(monkeypatch):
    z, i, t, v = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2)
    monkeypatch.setattr(q4, "_device_of", lambda *a: -1)         # lets tensors of the host past the first check
    for bad in ((z, i, [[0.0] * 3] * 2), (z, [[0] * 3] * 2, t), (z, i, None)):
        with pytest.raises(TypeError, match="torch.Tensor"):
            q4.qlora_distill_topk_fwd(*bad)
        with pytest.raises(TypeError, match="torch.Tensor"):
            q4.qlora_distill_topk_bwd(*bad, v, v)
