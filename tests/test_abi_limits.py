"""The largest sizes of the expert choice and of the 4-bit experts: refused on
the host by name, not by a failing launch (CPU only)."""
from test_abi_select_w4 import FAKE, INVALID, UNSUPPORTED, bwd, down, gate_up, lib, select  # noqa: F401


def test_tokens_of_the_choice(lib):  # noqa: F811
    """A block takes eight tokens, and their numbers are 32-bit."""
    for T in (2 ** 31 - 7, 2 ** 31 - 1):
        assert select(lib, T=T, k=1) == INVALID
        assert bwd(lib, T=T, k=1) == INVALID


def test_slots_of_the_4bit_experts(lib):  # noqa: F811
    """65535 rows of blocks, each of as many slots as its shared memory sorts:
    320 for 1024 experts, 2048 for one."""
    for E, k, row in ((1024, 8, 320), (1024, 3, 318), (1, 1, 2048)):
        T = 65535 * row // k
        for ids in (FAKE, None) if E == 1 else (FAKE,):
            assert gate_up(lib, T=T + 1, E=E, k=k, ids=ids) == UNSUPPORTED
            assert down(lib, T=T + 1, E=E, k=k, ids=ids, n=1 << 50) == UNSUPPORTED
