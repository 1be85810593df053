"""A context made on a side stream from memory that work queued there before still writes (GB300 only)."""
import pytest
import torch

from mixture_experts_ffn_router_gb300 import binding as B
from mixture_experts_ffn_router_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


@pytest.mark.parametrize("T", [64, 300])
def test_control_words_are_cleared_after_earlier_work(T):
    x = synth.make_x(T, seed=3, device="cuda")
    w = synth.make_weights(seed=4, device="cuda")
    early = B.MoeFFN(B.MOE_FFN_FULL_LAYER, T)
    want = early.forward(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block = torch.empty(early.nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        block.fill_(255)
        at = block.data_ptr()
        del block
        late = B.MoeFFN(B.MOE_FFN_FULL_LAYER, T)
        assert late.workspace.data_ptr() == at
        out = late.forward(x, w)
    torch.cuda.synchronize()
    assert late.status() == (B.MOE_FFN_OK, 0)
    assert torch.equal(out, want)
