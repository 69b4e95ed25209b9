"""The build refuses block-scaled 8-bit kernels of other registers than their warps share out (decided on ptxas's own lines)."""
import pytest

from ragged_grouped_gemm_02_gb300 import _build

ENTRY = """ptxas info    : Compiling entry function '%s' for 'sm_103a'
ptxas info    : Function properties for %s
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
"""
PAIR = "_ZN3rgg29grouped_fp8_block_pair_kernelILb1EEEvNS_6FpMapsENS_6FpArgsE"
WIDE = "_ZN3rgg24grouped_fp8_block_kernelILi1ELb0EEEvNS_6FpMapsENS_6FpArgsE"
NARROW = "_ZN3rgg24grouped_fp8_block_kernelILi2ELb0EEEvNS_6FpMapsENS_6FpArgsE"


def _log(pair, wide, narrow):
    return "".join(ENTRY % (name, name, n) for name, n in ((NARROW, narrow), (WIDE, wide), (PAIR, pair)))


def test_the_planned_registers():
    _build._check_registers(_log(96, 96, 168))


@pytest.mark.parametrize("registers", [(88, 96, 168), (96, 80, 168), (96, 96, 160), (104, 96, 168), (168, 96, 96)])
def test_others_are_refused(registers):
    with pytest.raises(RuntimeError, match="registers a thread"):
        _build._check_registers(_log(*registers))


def test_a_log_without_them():
    with pytest.raises(RuntimeError, match="no registers"):
        _build._check_registers("")
