"""What the build says about kernels that would be refused at run time."""
from video_vae_decoder_qkv_gb300 import build

REPORT = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN3abc16attention_kernelILb1ELi64ELi0EEEv14CUtensorMap_st' for 'sm_103a'
ptxas info    : Function properties for _ZN3abc16attention_kernelILb1ELi64ELi0EEEv14CUtensorMap_st
    8 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN3abc20attention_dkv_kernelILb0ELi128ELi3EEEv' for 'sm_103a'
ptxas info    : Used {} registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN3abc22attention_split_kernelILb0ELi1EEEv' for 'sm_103a'
ptxas info    : Used 96 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN3abc17join_parts_kernelILb1EEEv' for 'sm_103a'
ptxas info    : Used 47 registers, used 0 barriers
"""


def test_tile_kernels_of_the_launch_count_pass():
    assert build.refused_kernels(REPORT.format(168, 168)) == []
    assert build.refused_kernels("") == []


def test_others_are_named():
    found = build.refused_kernels(REPORT.format(160, 168))
    assert len(found) == 1 and "attention_kernel" in found[0] and "160 registers instead of 168" in found[0]
    assert len(build.refused_kernels(REPORT.format(166, 128))) == 2


def test_the_count_is_the_sources():
    with open(build.CSRC + "/h3qk_attn.cuh") as f:
        assert f"kLaunchRegs = {build.TILE_KERNEL_REGS}," in f.read()
