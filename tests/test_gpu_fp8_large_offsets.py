"""FP8 calls whose offsets pass 31 and 32 bits: the same 4096 rows over and over, 257 times, so that every row
of the large call has its bytes in a small one (the prologue's and the row operators' do not depend on the
batch) or, for the GEMM, in the call's own first rows, which are compared in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from bit_w4a4_quantized_group_b200 import binding as B
from bit_w4a4_quantized_group_b200 import build as BUILD

from gpu_helpers import check_device_error
from test_gpu_fp8_layer import _operand
from test_gpu_fp8_rows import _acts

pytestmark = pytest.mark.gpu

BLOCK, TIMES, K = 4096, 257, 2048
M = BLOCK * TIMES
assert M * K > 2 ** 31 and 2 * M * K > 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    BUILD.build()
    B.load()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _buffers(rows):
    sz = B.svdq_buffer_sizes("fp8", rows, 128, K, 0)
    return (torch.full((sz.a_codes,), 0xA5, dtype=torch.uint8, device="cuda"),
            torch.full((sz.a_scales,), 0xA5, dtype=torch.uint8, device="cuda"))


def _same_as_block(small, large):
    """Codes and scales (whole blocks of 128 rows) of every repetition are those of the small call."""
    check_device_error()
    for s, t in zip(small, large):
        t = t.view(TIMES, -1)
        assert t.shape[1] == s.numel()
        bad = [i for i in range(TIMES) if not torch.equal(t[i], s)]
        assert not bad, bad[:5]


@pytest.mark.parametrize("residual", [False, True])
def test_norm(residual):
    x, r = _acts(BLOCK, K, 1), _acts(BLOCK, K, 2) if residual else None
    small, large = _buffers(BLOCK), _buffers(M)
    h = torch.empty_like(x) if residual else None
    B.rmsnorm_quantize_act_t("fp8", x, r, None, 1e-6, h, *small)
    X, R = x.repeat(TIMES, 1), r.repeat(TIMES, 1) if residual else None
    B.rmsnorm_quantize_act_t("fp8", X, R, None, 1e-6, R, *large)             # H in the residual's place
    _same_as_block(small, large)
    if residual:
        assert all(torch.equal(t.view(torch.int16), h.view(torch.int16)) for t in R.view(TIMES, BLOCK, K))


@pytest.mark.parametrize("gated", [False, True])
def test_activation(gated):
    x = _acts(BLOCK, 2 * K if gated else K, 3)
    small, large = _buffers(BLOCK), _buffers(M)
    B.glu_quantize_act_t("fp8", "silu", x[:, :K], x[:, K:] if gated else None, None, *small)
    X = x.repeat(TIMES, 1)                                                   # with gating rows 2 K apart: 2^33 bytes
    B.glu_quantize_act_t("fp8", "silu", X[:, :K], X[:, K:] if gated else None, None, *large)
    _same_as_block(small, large)


@pytest.mark.parametrize("rank", [0, 32])
def test_prologue(rank):
    x, lam = _acts(BLOCK, K, 4), torch.linspace(0.5, 2.0, K, device="cuda")
    L1 = _acts(rank, K, 5) if rank else None
    small, large = _buffers(BLOCK), _buffers(M)
    z, Z = (torch.empty((n, rank), dtype=torch.bfloat16, device="cuda") if rank else None for n in (BLOCK, M))
    B.quantize_act_lowrank_down_t("fp8", x, lam, 1.0, L1, *small, z)
    B.quantize_act_lowrank_down_t("fp8", x.repeat(TIMES, 1), lam, 1.0, L1, *large, Z)
    _same_as_block(small, large)
    if rank:                    # K may be split otherwise: the repetitions agree, and differ from the block by roundings
        first = Z[:BLOCK]
        assert all(torch.equal(t.view(torch.int16), first.view(torch.int16)) for t in Z.view(TIMES, BLOCK, rank))
        xh = (x.float() / lam).to(torch.bfloat16).double()
        ref, S = xh @ L1.double().T, xh.abs() @ L1.double().abs().T
        assert ((first.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (K / 16 + 8) * 2.0 ** -23 * S).all()


@pytest.mark.parametrize("n,k,rank", [(128, 2048, 0), (2176, 128, 16)])
def test_gemm(n, k, rank):
    """Codes of A past 2^31 bytes, and Y past 2^32 bytes."""
    g = torch.Generator(device="cuda").manual_seed(k)
    a, sa, A = _operand(BLOCK, k, g, 2)
    w, sw, W = _operand(n, k, g, 2)
    z = (20.0 * torch.randn((BLOCK, rank), generator=g, device="cuda")).to(torch.bfloat16) if rank else None
    l2 = (20.0 * torch.randn((n, rank), generator=g, device="cuda")).to(torch.bfloat16) if rank else None
    Y = torch.full((M, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.w4a4_gemm_lowrank_up_t("fp8", M, n, k, rank, a.repeat(TIMES, 1), sa.repeat(TIMES), 1.0, w, sw, 1.0,
                             z.repeat(TIMES, 1) if rank else None, l2, None, Y)
    check_device_error()
    first = Y[:BLOCK]
    assert all(torch.equal(t.view(torch.int16), first.view(torch.int16)) for t in Y.view(TIMES, BLOCK, n))
    ref, S = A @ W.T, A.abs() @ W.abs().T
    if rank:
        ref, S = ref + z.double() @ l2.double().T, S + z.double().abs() @ l2.double().abs().T
    assert ((first.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (k / 32 + rank / 16 + 1) * 2.0 ** -23 * S).all()
