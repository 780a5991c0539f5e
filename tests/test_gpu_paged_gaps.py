"""Paged attention where a CTA's next unit is planned late: behind many requests without new tokens,
and behind requests whose units take long to add up."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from test_gpu_paged import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def run(b, arrays, only=None):
    ws = torch.zeros(int(sv.lib().spec_paged_attention_workspace_bytes(b.rows, b.H, b.Hk, b.D)),
                     dtype=torch.uint8, device=DEV)
    for _ in range(3):
        out, lse = sv.spec_paged_attention(b.q, *arrays, need_lse=True, workspace=ws)
        assert sv.spec_verify_device_status(ws) == sv.SPEC_OK
    b.check(out, lse, only=only)


def apart(b, gap):
    """The batch with ``gap`` requests without new tokens before each of its own."""
    n = len(b.sizes)
    new_start = b.new_start[:-1].repeat_interleave(gap + 1)
    new_start = torch.cat([new_start, b.new_start[-1:]])
    kv_len = torch.full((n, gap + 1), 40, dtype=torch.int32, device=DEV)
    kv_len[:, gap] = b.kv_len
    table = torch.full((n, gap + 1, b.table.shape[1]), -1, dtype=torch.int32, device=DEV)
    table[:, gap] = b.table
    return b.k, b.v, table.flatten(0, 1), new_start, kv_len.flatten()


SIZES = {
    "single tokens": [(1, 100 + i) for i in range(60)],
    "blocks": [(16, 60 + i) for i in range(60)],  # 64 rows of a head: one stream after the other
    "two streams": [(30, 90 + i) for i in range(40)],
    "all kinds": [x for i in range(12) for x in
                  ((1, 30 + i), (1, 260), (100, 140), (20, 30), (1, 1), (30, 41), (70, 200 + i), (2, 600))],
}


@pytest.mark.parametrize("gap", [1, 40, 300, 1500])
@pytest.mark.parametrize("kind", list(SIZES))
@pytest.mark.parametrize("D", [64, 128])
def test_units_behind_requests_without_new_tokens(D, kind, gap):
    b = Batch(SIZES[kind], Hk=8, G=4, D=D, P=32)
    assert (gap + 1) * len(b.sizes) <= 1 << 18
    run(b, apart(b, gap), only=set(range(0, len(b.sizes), 4)))


@pytest.mark.parametrize("first", [1, 5])
def test_single_tokens_before_a_long_chunk(first):
    b = Batch([(1, 20 + i) for i in range(first)] + [(9000, 9000)] + [(1, 90)] * 3, Hk=2, G=4, D=64, P=64)
    run(b, b.arrays(), only=set(range(first)) | {first + 1, first + 2})
    # (The chunk's rows against rows of a batch of its own.)
    r = slice(b.starts[first], b.starts[first + 1])
    out = sv.spec_paged_attention(b.q, *b.arrays())[r]
    start = torch.tensor([0, 9000], dtype=torch.int32, device=DEV)
    alone = sv.spec_paged_attention(b.q[r].contiguous(), b.k, b.v, b.table[first:first + 1].contiguous(),
                                    start, b.kv_len[first:first + 1].contiguous())
    # (Parts are cut elsewhere: sums rounded in another order, results to bfloat16 twice.)
    assert bool(((out.float() - alone.float()).abs() <= 2.0 ** -6 * (alone.float().abs() + 1.0)).all())
