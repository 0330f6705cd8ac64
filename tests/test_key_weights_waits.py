"""Every wait between the warps of the tcgen05 kernel of key_weights is bounded, and its
register split fits the launch: shown by reading its source, since a fault would hang the GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_15_gb300", "csrc")


def kernel():
    with open(os.path.join(CSRC, "key_weights_tc05.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read()).split("key_weights_tc05_kernel(", 1)[1]


def roles():
    return kernel().split("const uint32_t tmem = *tslot;", 1)[1].rsplit("__syncthreads();", 1)[0]


def test_waits_are_bounded_and_no_barrier_joins_warps():
    body = roles()
    assert "pt_wait(" in body and "mbar_try_wait(" not in body and "mbar_test_wait(" not in body
    for barrier in ("bar.sync", "bar.red", "barrier.", "__syncthreads", "bar.arrive"):
        assert barrier not in body, barrier


def test_the_loading_warp_waits_for_its_copies_on_every_way_out():
    role = roles().split("if (warp == 16) {", 1)[1].split("} else if (warp == 17", 1)[0]
    drain = role.index("mbar_wait(bar(S::B_UF + s)")
    before = role[:drain]
    assert "return;" not in role and before.count("{") - before.count("}") == 0  # under no condition of the role


def test_the_register_split_fits_the_launch():
    src = open(os.path.join(CSRC, "key_weights_tc05.cuh")).read()
    threads = int(re.search(r"kWtThreads = (\d+)", src).group(1))
    exp, other = (int(x) for x in re.search(r"kWtRegsExp = (\d+), kWtRegsOther = (\d+)", src).groups())
    assert threads == 640 and set(re.findall(r"reg_dec<(\w+)>", src)) == {"kWtRegsOther"}
    assert re.findall(r"reg_inc<(\w+)>", src) == ["kWtRegsExp"]
    launch = threads * (65536 // threads // 8 * 8)  # registers of the block at launch, eight at a time
    assert 512 * exp + 128 * other <= launch
