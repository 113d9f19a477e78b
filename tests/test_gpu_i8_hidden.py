"""Keys that a row of int8 attention does not see change none of its bits, in each kernel, where its references have moved."""
import pytest
import torch

import i8_bounds as bounds
from semi_ar_draft_gb300 import api, binding
from test_gpu_i8_attention import make_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kernel,G,Hk,D,n", [("few", 1, 4, 64, 4), ("few", 2, 2, 128, 4), ("few", 2, 1, 128, 4), ("few", 1, 1, 256, 8),
                                             ("few", 4, 2, 96, 2), ("rows", 4, 2, 128, 4), ("rows", 3, 1, 64, 5), ("wide", 16, 1, 128, 4),
                                             ("wide", 8, 2, 64, 8)])
def test_the_last_token_s_key_changes_no_other_row(dtype, kernel, G, Hk, D, n):
    """The last token's key and value, first of zeros and then far above all others, which makes its own row's references
    follow in the slice that the earlier tokens are in too.  Contexts of many slices a warp, so that theirs have settled."""
    lens = [6000 + 131 * j for j in range(24 // Hk)]
    c, lens, offsets = make_case(lens, [n] * len(lens), G * Hk, Hk, D, 64, 1, dtype, 3)
    assert bounds.kernel_of(c, n) == kernel
    outs = []
    for code, byte in ((0, 119), (127, 130)):
        for j, length in enumerate(lens):
            page, at = int(c["table"][j, (length - 1) // 64]), (length - 1) % 64
            last = c["q"][offsets[j + 1] - 1].view(Hk, G, D)[:, 0]  # a key along one of its queries
            c["codes"][0][page, at] = (torch.sign(last.float()) * code).to(torch.int8)
            c["codes"][1][page, at] = code
            for x in c["exps"]:
                x[page, :, at] = byte
        out, lse, ws = api.paged_attention_i8(c["q"], *c["codes"], *c["exps"], c["table"], c["seq"], c["offsets"], lse=True, max_new=n)
        assert binding.dspark_get_device_status(ws) == 0
        outs.append((out.view(len(lens), n, -1), lse.view(len(lens), n, -1)))
    for x, y in zip(*outs):
        assert torch.equal(x[:, :-1], y[:, :-1]) and not torch.equal(x[:, -1], y[:, -1])
