"""A decoding step as its documentation shows it, one row a sequence and no hint of how many: the kernel and the
workspace of single tokens."""
import pytest
import torch

from _kv import TYPES, Batch, rounded
from test_gpu_kv_attention import q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
def test_without_starts_every_sequence_has_one_row(q, kind, group):  # noqa: F811
    b = Batch([(1, 40 * n + 1) for n in range(40)], 2, 64, 16, seed=group, starts=False)
    cache, table, lengths, _ = b.device(q)
    x = torch.from_numpy(rounded(b.rng.standard_normal((b.rows, 2 * group, 64)), kind)).to(TYPES[kind]).cuda()
    hinted = q.qmm_kv_attention(x, cache, table, lengths, max_tokens=1)
    assert q.last_kernel() == "kv_attention_rows"
    size = q.qmm_kv_attention_workspace_bytes(b.rows, b.rows, 2 * group, 2, 64, TYPES[kind], max_tokens=1)
    small = torch.empty(size, dtype=torch.uint8, device="cuda")
    for args in (dict(), dict(workspace=small), dict(max_tokens=b.rows), dict(max_tokens=7, workspace=small)):
        y = q.qmm_kv_attention(x, cache, table, lengths, **args)
        assert q.last_kernel() == "kv_attention_rows", args
        assert torch.equal(y, hinted), args
    q.check_device_error()
    # what a call of its own takes is no more than it needs
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = q.qmm_kv_attention(x, cache, table, lengths)
    assert torch.cuda.max_memory_allocated() - before <= size + y.nbytes + 2048
