"""A Muon step that the host refuses leaves the momentum as it was: everything that can fail before a launch (kernel
attributes, tensor maps) comes before the first launch, the one that updates the momentum. By the order in the source:
no argument that passes the checks makes the driver refuse a map."""
import re

from moe_routing_swiglu_gb300 import _build

TEXT = re.sub(r"//[^\n]*", "", (_build.CSRC / "newton_schulz.cu").read_text())


def body(start):
    at = TEXT.index(start)
    return TEXT[at:TEXT.index("\n}\n", at)]


def test_the_products_have_their_maps_before_the_first_launch():
    f = body("cudaError_t launch_newton_schulz(")
    launch = f.index("launch_pre<float>")
    refusals = [m.start() for m in re.finditer(r"maps\.of\(|resident_pairs\(|device_status_ptr\(|cluster_shape\(", f)]
    assert len(refusals) == 11 and max(refusals) < launch
    # a launch only looks its maps up: every operand and box that one asks for is among them
    assert set(re.findall(r"maps\.of\((\w+), (\w+)\)", f)) == {
        ("x", "gram_box"), ("x", "apply_box"), ("next", "gram_box"), ("next", "apply_box"), ("a", "BM"), ("b", "BM"),
        ("t", "BM"), ("b1", "BM")}
    assert "enc(" not in f and TEXT.count("enc(&") == 2


def test_the_one_launch_way_sets_its_attributes_first():
    f = body("cudaError_t launch_cluster(")
    assert max(m.start() for m in re.finditer("cudaFuncSetAttribute", f)) < f.index("launch_squares<")
    assert f.index("launch_squares<") < f.index("cudaLaunchKernelEx")
