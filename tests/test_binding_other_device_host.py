"""A status word on another device is refused by the page planning, shared-latent and prompt calls
before any CUDA call: their kernels run on the current device and would write to it from there."""
import pytest
import torch

import decode_attention_stief_b200 as stief


class _OnAnotherDevice:
    """What the binding looks at of a status word on the second GPU."""
    dtype, is_cuda, device = torch.int32, True, "cuda:1"

    def numel(self):
        return 1

    def get_device(self):
        return 1

    def data_ptr(self):
        return 0x10000


@pytest.mark.parametrize("name,nargs", [("stief_plan_pages", 12), ("stief_append_shared_paged", 4),
                                        ("stief_decode_shared_paged", 8), ("stief_expand_shared_paged", 7),
                                        ("stief_prefill_attention", 8)])
def test_status_word_on_another_device(name, nargs):
    with pytest.raises(ValueError, match="dev_status must be on the current device"):
        getattr(stief, name)(*[64] * nargs, dev_status=_OnAnotherDevice())
