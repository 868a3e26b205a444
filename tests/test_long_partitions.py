"""Partitions longer than any context are one partition, however long: sizes here,
results on the GPU."""
import pytest
import torch

HUGE = 2 ** 31 - 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_224_gb300 import build
    build.build()


def test_sizes():
    import paged_kv_cache_224_gb300 as pa
    assert pa.pa_decode_workspace_bytes(4, 8, 2, 128, 16, 1000, HUGE) == 0
    assert pa.pa_decode_shared_prefix_workspace_bytes(4, 4, 4, 128, 16, 1000, 2, HUGE) == \
        pa.pa_decode_shared_prefix_workspace_bytes(4, 4, 4, 128, 16, 1000, 2, 1008) > 0
    assert pa.pa_decode_partition_tokens(4, 8, 2, 16, 1000, HUGE) == HUGE       # as given


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (8, 1, 128), (4, 4, 64)])
def test_results(Hq, Hkv, D):
    import paged_kv_cache_224_gb300 as pa
    from tests.helpers import check_attention, to_f64
    from tests.ref64 import attend, gather, make_pool
    dev = torch.device("cuda:0")
    lens = [1000, 1, 0, 300]
    kc, vc, bt, _ = make_pool(lens, Hkv, D, 16, "bf16", dev, 1)
    q = torch.randn((4, Hq, D), generator=torch.Generator().manual_seed(2)).bfloat16().to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    ref = torch.stack([attend(q[s].cpu().double(), gather(kc, bt[s], L), gather(vc, bt[s], L), 0.1)[0] for s, L in enumerate(lens)])
    out = torch.full_like(q, float("nan"))
    pa.pa_decode(out, q, kc, vc, bt, n, 0.1, 1000, HUGE)
    check_attention(to_f64(out), ref.numpy(), "bf16", "decode")
    if Hq // Hkv <= 4:   # two samples behind 16 tokens of the first sequence
        bt2 = bt[:1].repeat(2, 1).contiguous()
        out = torch.full_like(q[:2], float("nan"))
        pa.pa_decode_shared_prefix(out, q[:2].contiguous(), kc, vc, bt2, n[:1].repeat(2), 0.1, 1000, 2, 1, HUGE)
        ref = torch.stack([attend(q[s].cpu().double(), gather(kc, bt[0], 1000), gather(vc, bt[0], 1000), 0.1)[0] for s in range(2)])
        check_attention(to_f64(out), ref.numpy(), "bf16", "shared prefix")
