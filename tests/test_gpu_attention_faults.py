"""The block attention's give-up path: its bounded waits run out on purpose (needs a B200).

uno_attention_test_hook (a test-only hook of the C ABI) leaves the queries of all
but the first few parts of each CTA unannounced. The MMA issuer and the softmax warps
that wait for them give up after a second, the other roles after them. The kernels
must still exit normally, the rows that were not completed must be NaN (the second
launch reads only what an item's entry allows, whatever the workspace held), all
other rows must be as without the hook, and the call that follows is correct and
sets no bit.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PRODUCER, MMA, SOFTMAX = 8, 16, 32


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    from lossless_decoding_b200 import api as A
    return A


# query rows of one to 16, 32, 64 and 136: every layout of a tile
@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (1, 7, 64), (1, 16, 128), (8, 4, 64),
                                   (16, 4, 128), (17, 8, 128)])
def test_waits_run_out_and_incomplete_rows_are_nan(api, T, G, D):
    from lossless_decoding_b200._lib import lib
    B, H, page = 200, 4, 128
    g = torch.Generator(device=DEV).manual_seed(T * G + D)
    c = api.kv_cache(torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1), B, H, page, D)
    for codes in (c.k, c.v):
        codes.copy_(torch.randn(codes.shape, generator=g, device=DEV))
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    q, k, v = (torch.randn(B, T, h, D, generator=g, device=DEV).bfloat16()
               for h in (H * G, H, H))
    lens = torch.full((B,), 100, dtype=torch.int32, device=DEV)
    clean = api.block_attention(q, k, v, c, lens)
    assert torch.isfinite(clean).all() and api.device_fault_flags() == 0
    # items of one tile, dealt out evenly: some CTAs have this many, the others one more
    items = B * H * -(-T * G // 128)
    segments = items // torch.cuda.get_device_properties(0).multi_processor_count
    need = int(lib.uno_block_attention_workspace_bytes(B, T, H * G, H, D))
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV)
    assert lib.uno_attention_test_hook(segments) == 0
    try:
        out = api.block_attention(q, k, v, c, lens, workspace=ws)
        torch.cuda.synchronize()  # the kernels returned: no hang, no device fault
        flags = api.device_fault_flags()
    finally:
        assert lib.uno_attention_test_hook(0) == 0
    assert flags & MMA and flags & SOFTMAX, f"flags {flags:#x}"
    # a sequence's and KV head's rows of a row tile stand or fall together
    lost = torch.isnan(out).view(B, T, H, G, D)
    assert lost.any() and not lost.all()
    assert torch.equal(lost, lost[..., :1].expand_as(lost))
    keep = ~lost.view_as(out)
    assert torch.equal(out[keep], clean[keep])
    again = api.block_attention(q, k, v, c, lens, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(again, clean) and api.device_fault_flags() == 0
