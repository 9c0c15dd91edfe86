"""Operands that do not belong together are refused by the low-precision bindings before
anything is enqueued (host tensors here; the device check and the launch are stood in for)."""
import pytest

torch = pytest.importorskip("torch")
import post_weight_quantization_22_amd as gq  # noqa: E402
from post_weight_quantization_22_amd import _lib  # noqa: E402

T, M, N = 5, 300, 272
MB, NB = 3, 3
U8, BF, F32 = torch.uint8, torch.bfloat16, torch.float32


@pytest.fixture
def launched(monkeypatch):
    with pytest.raises(ValueError):
        _lib._on_gpu(torch.zeros(1), "t")  # fills the dtype table
    calls = []
    monkeypatch.setattr(_lib, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(_lib, "_launch", lambda name, *a: calls.append(name))
    monkeypatch.setattr(_lib, "_space", lambda need, ws, device, stream: (None, 0, None))
    return calls


def _z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def _refused(launched, f, good, **changes):
    """good runs; each change of one argument is refused."""
    f(**good)
    assert len(launched) == 1
    for name, values in changes.items():
        for v in values:
            with pytest.raises(ValueError, match=name):
                f(**{**good, name: v})
    assert len(launched) == 1


def test_gemm(launched):
    good = dict(X=_z(T, N, dtype=U8), xscales=_z(NB, T), W=_z(M, N, dtype=U8), wscales=_z(MB, NB),
                Y=_z(T, M), residual=_z(T, M))
    _refused(launched, gq.fp8_gemm, good,
             W=[_z(M, N + 16, dtype=U8), _z(M, N - 16, dtype=U8)],
             xscales=[_z(NB + 1, T), _z(NB, T - 1)],
             wscales=[_z(MB + 1, NB), _z(MB, NB + 1), _z(MB - 1, NB)],
             residual=[_z(T + 1, M), _z(T, M + 1)],
             Y=[_z(T, M - 1), _z(T - 1, M)])
    # outputs, a residual in place and scales of more tokens may be larger
    Y = _z(T + 1, M + 8)
    gq.fp8_gemm(**{**good, "Y": Y, "residual": Y, "xscales": _z(NB, T + 3)})
    assert len(launched) == 2


def test_linear(launched):
    good = dict(X=_z(T, N, dtype=BF), W=_z(M, N, dtype=U8), wscales=_z(MB, NB), Y=_z(T, M))
    _refused(launched, gq.fp8_linear, good,
             W=[_z(M, 2 * N, dtype=U8), _z(M, N - 16, dtype=U8)],
             wscales=[_z(MB, 2 * NB), _z(MB + 1, NB)])


def test_gated(launched):
    good = dict(X=_z(T, N, dtype=U8), xscales=_z(NB, T), Wg=_z(M, N, dtype=U8), gscales=_z(MB, NB),
                Wu=_z(M, N, dtype=U8), uscales=_z(MB, NB), codes=_z(T, M, dtype=U8), scales=_z(MB, T))
    _refused(launched, gq.fp8_gated_gemm, good,
             Wu=[_z(M + 1, N, dtype=U8), _z(M, N + 16, dtype=U8), _z(M - 1, N, dtype=U8)],
             Wg=[_z(M, N + 16, dtype=U8)],
             gscales=[_z(MB + 1, NB)], uscales=[_z(MB, NB + 1)], xscales=[_z(NB + 1, T)])


def test_swiglu(launched):
    good = dict(gate=_z(T, N), up=_z(T, N), codes=_z(T, N, dtype=U8), scales=_z(NB, T))
    _refused(launched, gq.fp8_swiglu_quantize, good, up=[_z(T + 1, N), _z(T, N + 1), _z(T, N - 1)])
