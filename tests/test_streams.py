"""Calls on another stream than the current one (`stream=`): memory that a call allocates for itself."""
import contextlib

import pytest
import torch

import bit_nf4_quantized_23_b200 as q4

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_nf4_quantized_23_b200.build import build
    build()


M, N, K, R, ADS, V, TOP = 5, 48, 128, 8, 2, 40, 3


def calls(w, z):
    """Each entry point that allocates, with zeros of the right shapes from z(shape, dtype); by name."""
    X, dY, A, B = z((M, K), BF16), z((M, N), BF16), z((R, K), BF16), z((N, R), BF16)
    A_all, B_all, idx, scales = z((ADS, R, K), BF16), z((ADS, N, R), BF16), z((M,), I32), z((ADS,), F32)
    logits, t_idx, t = z((M, V), F32), z((M, TOP), I32), z((M, TOP), F32)
    codes, alpha = z((256,), torch.int8), z((4,), F32)
    return {
        "quantize": lambda **k: q4.qlora_quantize_nf4_dq(z((N, K), BF16), **k),
        "dequantize": lambda **k: q4.qlora_dequantize(w, **k),
        "quantize_int8": lambda **k: q4.qlora_quantize_int8_absmax(z((256,), BF16), **k),
        "dequantize_int8": lambda **k: q4.qlora_dequantize_int8_absmax(codes, alpha, **k),
        "merge": lambda **k: q4.qlora_merge_lora(w, A, B, R, 16.0, **k),
        "fwd": lambda **k: q4.qlora_linear_fwd(w, X, A, B, R, 16.0, **k),
        "fwd_multi": lambda **k: q4.qlora_linear_fwd_multi(w, X, A_all, B_all, idx, R, 16.0, save_U=True, **k),
        "bwd": lambda **k: q4.qlora_linear_bwd(w, X, dY, A, B, R, 16.0, **k),
        "fwd_adapters": lambda **k: q4.qlora_linear_fwd_adapters(w, X, A_all, B_all, idx, scales, **k),
        "bwd_adapters": lambda **k: q4.qlora_linear_bwd_adapters(w, X, dY, A_all, B_all, idx, scales, **k),
        "distill_fwd": lambda **k: q4.qlora_distill_topk_fwd(logits, t_idx, t, **k),
        "distill_bwd": lambda **k: q4.qlora_distill_topk_bwd(logits, t_idx, t, z((M,), F32), z((M,), F32), **k),
    }


class FakeStream:
    def __init__(self, at):
        self.cuda_stream = at


@pytest.mark.parametrize("name", sorted(calls(None, lambda s, d: torch.zeros(s, dtype=d))))
def test_what_a_call_allocates_belongs_to_its_stream(name, monkeypatch):
    """On the host: the caching allocator gives a freed block to the next request of the stream that it was
    allocated on, so a workspace that the kernels of `stream` use has to be allocated on that stream, and so
    have the outputs, which the current stream uses as well."""
    real, on, allocated, recorded, launched = q4.lib(), [], [], [], []

    class Library:
        def __getattr__(self, f):
            if f.endswith(("_size", "_sizes")):
                return getattr(real, f)
            return lambda *a: launched.append(a) or 0

    @contextlib.contextmanager
    def stream_context(s):
        on.append(s)
        yield
        on.pop()

    empty = torch.empty

    def counted(*a, **k):
        allocated.append((on[-1] if on else None, empty(*a, **k)))
        return allocated[-1][1]

    w = q4.NF4Weight.empty(N, K, device="cpu")
    call = calls(w, lambda s, d: torch.zeros(s, dtype=d))[name]
    monkeypatch.setattr(q4, "lib", Library)
    monkeypatch.setattr(q4, "_need", lambda *a: None)
    monkeypatch.setattr(q4, "_device_of", lambda *a: -1)
    monkeypatch.setattr(q4, "_raw_stream", None)
    monkeypatch.setattr(torch, "empty", counted)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    current, s = FakeStream(3), FakeStream(7)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at: s if at == 7 else None)
    got = call(stream=s)
    assert allocated and len(launched) == 1
    assert all(at is s for at, _ in allocated)
    if isinstance(got, q4.NF4Weight):
        got = [getattr(got, b) for b in got._BUFFERS]
    returned = [t for t in (got if isinstance(got, (tuple, list)) else (got,)) if t is not None]
    assert sorted(p for p, _ in recorded) == sorted(t.data_ptr() for t in returned)
    assert all(by is current for _, by in recorded)
    # the current stream, named or not: allocated as ever
    for same in (dict(), dict(stream=current)):
        allocated.clear(), recorded.clear()
        call(**same)
        assert allocated and all(at is None for at, _ in allocated) and not recorded


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [16, 100, 700])
def test_calls_on_other_streams_beside_the_current_one(tokens):
    """Two streams that are still busy when the calls return, their workspaces left to the call, while the
    current stream allocates and overwrites blocks of the same sizes."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    n, k, r = 520, 512, 16
    w = q4.qlora_quantize_nf4_dq(rnd(n, k))
    sets = [(rnd(tokens, k), rnd(tokens, n), rnd(4, r, k), rnd(4, n, r),
             torch.randint(-1, 4, (tokens,), generator=g, device="cuda").int()) for _ in range(2)]
    scales = torch.ones(4, device="cuda")
    size = max(q4.qlora_adapters_workspace_size(tokens, n, k, r, 4), q4.qlora_linear_workspace_size(tokens, n, k, r))

    def run(x, stream):
        X, dY, A, B, idx = x
        Y, U = q4.qlora_linear_fwd_adapters(w, X, A, B, idx, scales, stream=stream)
        got = (Y, U) + q4.qlora_linear_bwd_adapters(w, X, dY, A, B, idx, scales, U_saved=U, stream=stream)
        Y, U = q4.qlora_linear_fwd(w, X, A[0], B[0], r, 16.0, stream=stream)
        return got + (Y, U) + q4.qlora_linear_bwd(w, X, dY, A[0], B[0], r, 16.0, U_saved=U, stream=stream)

    want = [run(x, None) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, x in zip(streams, sets):
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)                     # about a millisecond
            got.append(run(x, s))
        for _ in range(8):
            torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(want, got):
            for u, v in zip(a, b):
                assert torch.equal(u, v)
    torch.cuda.synchronize()
    assert q4.qlora_read_device_errors(clear=True) == 0
