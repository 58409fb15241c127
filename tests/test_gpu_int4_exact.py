"""4-bit products whose every sum is exact in fp32, so that a lost column, a
nibble out of order or a scale of another group shows in any order of sums.

Activations are whole numbers up to 4, scales 1/2, 1 or 2.  The sums of a group
hold 1.5 x and q x / 16: multiples of 2^-4 below 128 x 4 x 3.44 < 2^11.  Scaled
and added up they are multiples of 2^-5, at most 4 x 8 / 16 x 2 = 4 per column,
below 2^17 for 16512 columns: 22 bits, and fp32 holds 24."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def A():
    from routed_expert_int4_amd import attention
    return attention


def case(M, N, K, group):
    assert K <= 16512
    g = torch.Generator(device=DEV).manual_seed(M + N + K + group)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scale = 2.0 ** torch.randint(-1, 2, (N, K // group), generator=g, device=DEV)
    low, high = codes.int() & 15, codes.int() >> 4
    q = torch.stack([low, high], 2).flatten(1)
    w = torch.where(q > 7, q - 16, q).double() * scale.double().repeat_interleave(group, 1)
    return x, codes, scale.half(), x.double() @ w.t()


def check(A, M, N, K, group):
    x, codes, scale, want = case(M, N, K, group)
    assert torch.equal(A.int4_linear(x, codes, scale, out_dtype=torch.float32).double(), want)
    assert torch.equal(A.int4_linear(x, codes, scale), want.bfloat16())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2])
@pytest.mark.parametrize("N,K", [(7, 128), (33, 8192), (17, 8320), (40, 8576), (16, 16512)])
def test_dot_products(A, M, N, K, group):
    """Segments of 256 columns and turns of 8192, whole and begun."""
    check(A, M, N, K, group)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [3, 16, 17, 32])
@pytest.mark.parametrize("N,K", [
    (100, 2176), (100, 8192), (100, 8320), (7, 16512),  # eight waves, 16 weight rows: turns of 8192 columns
    (4100, 2304), (4100, 8320),                         # eight waves, 32 rows
    (50, 128), (50, 2048), (8200, 4096), (8200, 4224),  # four waves, 16 rows: turns of 4096
    (12300, 128), (12300, 4224),                        # four waves, 32 rows
])
def test_up_to_32_tokens(A, M, N, K, group):
    check(A, M, N, K, group)


SHAPES = [  # tokens x weight rows of a tile, and columns of a stage
    (33, 70),      # 32 x 32, 512
    (64, 4100),    # 32 x 64, 256
    (130, 4100),   # 64 x 64, 256
    (256, 6144),   # 64 x 128, 128
    (1025, 6150),  # 128 x 128, 64
    (1000, 4100),  # 128 x 192, 64
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [384, 8320])
@pytest.mark.parametrize("M,N", SHAPES)
def test_more_tokens(A, M, N, K, group):
    """Stages whole and begun, turns of 8192 columns, tiles cut by either edge."""
    check(A, M, N, K, group)


@pytest.mark.parametrize("K,group", [(160, 32), (8224, 32), (8256, 64)])
@pytest.mark.parametrize("M,N", SHAPES)
def test_stages_that_end_early(A, M, N, K, group):
    check(A, M, N, K, group)


@pytest.mark.parametrize("M", [1, 2, 3, 16, 17, 32])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 64), (96, 32), (160, 32), (192, 64), (1056, 32), (4128, 32), (8224, 32), (8256, 64)])
def test_columns_that_end_early(A, M, K, group):
    check(A, M, 70, K, group)
