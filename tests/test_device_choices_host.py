"""What the library keeps per shape is kept per device: a process that uses a second device with another number of SMs
gets that device's choices, and the first one's again when it goes back. (Host code; the test hook names the device.)"""

SHAPES = [(100, 4096, 1000), (333, 4112, 1003), (16, 4096, 14336), (512, 4096, 14336), (2048, 4096, 14336)]


def test_plans_follow_the_device():
    import bit_weight_only_pack_b200 as lbq
    plans = {}
    try:
        for dev, sms in ((61, 148), (62, 24), (61, 148), (63, 148)):
            lbq.lbq_debug_device(dev, sms)
            got = [lbq.lbq_debug_w8a8_planned(*s) for s in SHAPES]
            assert plans.setdefault(sms, got) == got
    finally:
        lbq.lbq_debug_device(-1, 0)
    assert plans[24] != plans[148]
