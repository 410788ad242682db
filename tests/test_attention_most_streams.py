"""Rows of as many streams as a call takes, into 8-bit pages."""
import pytest

from tests.helpers import say

pytestmark = pytest.mark.gpu


def test_the_most_streams_write_their_rows_in_8_bits():
    """Every row comes back as it was written, within half a code and the rounding to bf16, and no other place is touched."""
    import torch

    import byte_level_lm_amd as B
    n, h, d, page = 65535, 24, 16, 16
    gen = torch.Generator(device="cuda").manual_seed(9)
    pools = [torch.full((n, h, page, d), 99, device="cuda", dtype=torch.int8) for _ in range(2)]
    sc = {x: torch.full((n, h, page), 7.0, device="cuda") for x in ("k_scale", "v_scale")}
    table = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)[:, None].contiguous()
    k, v = (torch.randn(n, h, d, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in range(2))
    start = torch.randint(0, page, (n,), device="cuda", generator=gen, dtype=torch.int32)
    say("8-bit write of", n, "streams")
    B.kv_write(k, v, *pools, table, start=start, **sc)
    back = B.kv_read(*pools, table, torch.arange(n + 1, device="cuda"), n, start=start, **sc)
    there = torch.arange(page, device="cuda")[None] == start[table[:, 0].long().argsort()].long()[:, None]  # [pages, places]
    at = (table[:, 0].long(), start.long())
    for x, got, pool, scale in zip((k, v), back, pools, sc.values()):
        top = x.float().abs().amax(-1, keepdim=True)
        assert torch.all((got.float() - x.float()).abs() <= 1.01 * top * (0.5 / 127 + 2.0 ** -8))
        assert torch.all((scale[at[0], :, at[1]] - top[..., 0] / 127).abs() <= 2.0 ** -22 * top[..., 0] / 127)
        rest = ~there[:, None, :].expand(-1, h, -1)
        assert torch.all(pool[rest] == 99) and torch.all(scale[rest] == 7.0)
