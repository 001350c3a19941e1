"""The binding's constants are the header's."""
import os
import re

import combine_ep_get_amd as ep

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep_get.h")


def test_binding_constants_match_the_header():
    with open(HEADER) as f:
        defines = dict(re.findall(r"^#define (EP_[A-Z]\w*) +([^/\n]+)", f.read(), re.M))
    names = {n for n in dir(ep) if re.match(r"EP_[A-Z]", n)} & set(defines)
    assert {"EP_MOE_TOKENS_MAX", "EP_MAX_FEATURES", "EP_ACT_GEGLU", "EP_MAX_TOPK", "EP_ERR_HIP"} <= names
    for n in names:
        minus, value, shift = re.fullmatch(r"\(?(-?)(\d+)u?(?: << (\d+))?\)?", defines[n].strip()).groups()
        assert getattr(ep, n) == (-1 if minus else 1) * int(value) << int(shift or 0), n
