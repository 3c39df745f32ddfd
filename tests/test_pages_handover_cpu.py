"""The tiered cache's binding refuses fp16 before anything else is looked at (no GPU needed)."""
import numpy as np
import pytest


@pytest.mark.parametrize("lib", ["torch", "numpy"])
def test_fp16_is_refused(lib):
    import tiered_quantize_evict_gb300 as qe
    if lib == "torch":
        torch = pytest.importorskip("torch")
        half, good = torch.zeros(8, dtype=torch.float16), [torch.zeros(8, dtype=t) for t in (torch.bfloat16, torch.int16, torch.float32)]
    else:
        half, good = np.zeros(8, np.float16), [np.zeros(8, t) for t in (np.uint16, np.int16, np.float32)]
    for _ in range(2):
        with pytest.raises(qe.QEError, match="k is fp16"):
            qe._bf16("k", half)
    assert [qe._bf16("k", x) == qe._ptr(x) for x in good] == [True] * 3
