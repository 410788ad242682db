"""Windows beside prefixes that are long: the host does not know how long, and may not take them for short where few workgroups
would read them."""
import pytest

from tests.helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("streams,heads,d,q8", [(32, 8, 64, True), (64, 4, 32, False)])
def test_a_window_behind_a_long_prefix_is_no_slower_than_no_window(streams, heads, d, q8):
    """Prefix and window together are all positions, as without a window."""
    import torch

    import byte_level_lm_amd as B
    n, page = 32768, 64
    gen = torch.Generator(device="cuda").manual_seed(d)
    shape = (streams * n // page, heads, page, d)
    if q8:
        pages = [torch.randint(-127, 128, shape, device="cuda", generator=gen, dtype=torch.int8) for _ in range(2)]
        scales = {x: torch.full(shape[:3], 1 / 64, device="cuda") for x in ("k_scale", "v_scale")}
        most = 127 / 64
    else:
        pages, scales = [torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16) for _ in range(2)], {}
        most = float(pages[1].abs().max())
    table = torch.randperm(shape[0], device="cuda", generator=gen).to(torch.int32).view(streams, -1)
    q = torch.randn(streams, heads, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    lengths = torch.full((streams,), n, device="cuda", dtype=torch.int32)
    prefix = torch.full((streams,), n - 512, device="cuda", dtype=torch.int32)
    calls = {"window": lambda: B.attention_step(q, *pages, table, lengths, window=512, prefix=prefix, **scales),
             "none": lambda: B.attention_step(q, *pages, table, lengths, **scales)}
    out = {x: f().float() for x, f in calls.items()}
    # each is off by the rounding to bf16, 2^-16 twice of the mean |v| by its weights, and less than that by the rest
    assert torch.all((out["window"] - out["none"]).abs() <= 2.0 ** -7 * out["none"].abs() + 2.0 ** -13 * most)
    ms = {x: [] for x in calls}
    for _ in range(7):
        for x, f in calls.items():
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            f()
            a.record()
            for _ in range(5):
                f()
            b.record()
            torch.cuda.synchronize()
            ms[x].append(a.elapsed_time(b) / 5)
    took = {x: sorted(t)[3] for x, t in ms.items()}
    say("window behind a prefix", took, "ms")
    assert took["window"] < 1.4 * took["none"]
