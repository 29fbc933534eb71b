"""Kernels that redistribute their registers are checked when they are built: one
that got fewer than it hands out would wait for ever."""
import pytest

from atomistic_mlip_b200 import build as build_mod


def _report(name, regs):
    return (f"ptxas info    : Compiling entry function '{name}' for 'sm_100a'\n"
            f"ptxas info    : Function properties for {name}\n    0 bytes stack frame, 0 bytes spill stores\n"
            f"ptxas info    : Used {regs} registers, used 1 barriers, 1024 bytes smem\n")


REG = "_ZN3e2f3lin3reg15gemm_reg_kernelIfLb0ELb0ELi1ELb1EEEvNS1_4ArgsE"
TMA = "_ZN3e2f3lin3tma15gemm_tma_kernelILb0ELb0ELi{}ELb{}ELi3ELi8ELb0EEEv14CUtensorMap_st"


def test_too_few_registers_end_the_build():
    assert build_mod.check_registers(_report(REG, 72) + _report(TMA.format(128, 1), 168)) == 2
    assert build_mod.check_registers(_report(REG, 70) + _report(TMA.format(256, 1), 162)) == 2   # launched with 72, 168
    assert build_mod.check_registers(_report(TMA.format(256, 0), 90) + _report("other", 20)) == 0
    for bad in (_report(REG, 64), _report(TMA.format(256, 1), 160), _report("other", 20) + _report(REG, 40)):
        with pytest.raises(RuntimeError):
            build_mod.check_registers(bad)


def test_the_names_are_those_of_the_sources():
    src = {n: open(f"{build_mod.CSRC}/{n}.cu").read() for n in ("linear_reg", "linear_tma")}
    assert "gemm_reg_kernel(" in src["linear_reg"] and "LAUNCH_REGS = 72" in src["linear_reg"]
    assert "template <bool AMN, bool BMN, int BN, bool LONGK, int EPI, int EW, bool IO" in src["linear_tma"]
    assert "gemm_tma_kernel(" in src["linear_tma"] and "LONGK ? 168 : 0" in src["linear_tma"]
