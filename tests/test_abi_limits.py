"""The largest sizes of the 4-bit experts: refused on the host by name, not by a
failing launch (CPU only)."""
from test_abi_select_w4 import FAKE, UNSUPPORTED, down, gate_up, lib  # noqa: F401


def test_slots_of_the_4bit_experts(lib):  # noqa: F811
    """65535 rows of blocks, each of as many slots as its shared memory sorts:
    320 for 1024 experts, 2048 for one."""
    for E, k, row in ((1024, 8, 320), (1024, 3, 318), (1, 1, 2048)):
        T = 65535 * row // k
        for ids in (FAKE, None) if E == 1 else (FAKE,):
            assert gate_up(lib, T=T + 1, E=E, k=k, ids=ids) == UNSUPPORTED
            assert down(lib, T=T + 1, E=E, k=k, ids=ids, n=1 << 50) == UNSUPPORTED
