"""How many workgroups the router losses' first launch has, read from the size of
the workspace that they write partial rows to (host only): none without a row of
logits, and one without a second launch for batches of four rounds."""
import pytest

from mixture_experts_routed_amd import abi


def workspace(blocks, E):
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    join = -(-E // 16)
    return 2 * up(blocks * E * 4) + 2 * up(blocks * 4) + 2 * up(join * 4) + up(4)


# rows of a workgroup: 1,024 threads, 8 to 64 lanes a row (16 for 9 to 32 experts whose
# rows are not whole 16-byte chunks; the logits' address may make them so for any E)
@pytest.mark.parametrize("E,rows", [(1, 128), (8, 128), (9, 64), (17, 64), (32, 64), (33, 64),
                                    (60, 64), (64, 64), (65, 32), (128, 32), (129, 16), (512, 16),
                                    (1024, 16)])
def test_every_workgroup_has_a_row(E, rows):
    one = 4 * (128 if E <= 32 else rows)
    for T in (1, one, one + 1, 1000, 4000, 5000, 256 * rows, 256 * rows + 1, 40000):
        blocks = 1 if T <= one else min(256, -(-T // rows))
        assert abi.moe_balance_workspace(T, E, 1) == workspace(blocks, E), (T, blocks)
